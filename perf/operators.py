"""Cases for the operators of a block-scaled 8-bit K/V cache (``H2OBlockCache``).

A cache holds, for each sequence and cached head, up to ``capacity`` entries of
d codes for K and for V (e4m3 or int8) with one power-of-two scale for each
block of 32 entries, a position tag and an accumulated attention weight.

  fill     new K/V rows quantised and appended (the prompt, or a chunk of it)
  step     decode: the new tokens appended, then their queries attend over the
           cache and every entry's weight is added to its score
  attend   queries over a cache that stays as it is (an encoder's states)
  evict    every sequence cut down to k_heavy + k_local entries by its scores

``run`` computes them in elementary torch operations, or with the framework's
calls where ``own`` is set; ``exact`` computes them in 64 bits, one sequence at
a time, from the definitions."""
import math

import torch

own = False

BLOCK = 32                               # entries that share a scale
LIMIT = {"e4m3": 448.0, "int8": 127.0}   # largest code
STORE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MIN_EXP = -100                           # smallest scale: 2^-100


def listed():
    case = dict(kv="e4m3", d=128, G=1, n=1, ragged_counts=False, causal=True, accumulate=True, tokens_first=False)
    return [
        # one sequence of 32 heads at a small budget: latency
        dict(case, name="step one sequence", kind="step", B=1, H=32, lo=255, hi=255),
        # eight sequences of an OPT-6.7B-shaped layer, their whole text still cached
        dict(case, name="step 32 heads", kind="step", B=8, H=32, lo=2559, hi=2559),
        # an OPT-30B-shaped layer, sequences of every age in one batch
        dict(case, name="step 56 heads ragged", kind="step", kv="int8", B=64, H=56, lo=700, hi=2047),
        # grouped queries: four query heads share a cached one; odd lengths; fused projection's token-first rows
        dict(case, name="step groups of 4", kind="step", kv="int8", B=16, H=8, G=4, lo=3001, hi=8447, tokens_first=True),
        # draft tokens verified: up to five queries a sequence, not the same number for each
        dict(case, name="step draft tokens", kind="step", B=8, H=8, G=8, n=5, d=64, lo=1000, hi=8100,
             ragged_counts=True, tokens_first=True),
        # one long text, groups of eight
        dict(case, name="step long", kind="step", B=1, H=8, G=8, lo=262000, hi=262000),
        # a decoder's queries over encoder states of another length, some sequences without any
        dict(case, name="attend encoder states", kind="attend", kv="int8", B=12, H=16, d=64, n=7, lo=0, hi=1500,
             causal=False, accumulate=False),
        # a prompt of 8K tokens
        dict(case, name="fill prompt", kind="fill", B=16, H=32, n=8192, lo=0, hi=0, tokens_first=True),
        # chunks of different lengths appended behind what is there, blocks partly filled
        dict(case, name="fill chunk", kind="fill", kv="int8", d=64, B=3, H=8, n=77, lo=1, hi=100, ragged_counts=True),
        # the 8K-prompt cache cut down to a 20 % budget
        dict(case, name="evict 8K", kind="evict", B=32, H=32, lo=8448, hi=8448, k_heavy=845, k_local=845, n_sink=0,
             score_mode=0),
        # a small ragged batch, some rows within the budget; ranked by mean weight, first positions pinned
        dict(case, name="evict small", kind="evict", kv="int8", d=64, B=5, H=8, lo=100, hi=700, k_heavy=64, k_local=65,
             n_sink=4, score_mode=1),
        # one long text
        dict(case, name="evict long", kind="evict", B=1, H=8, lo=131072, hi=131072, k_heavy=13107, k_local=13107,
             n_sink=0, score_mode=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "step", "step", "attend", "fill", "evict"])
    c = dict(kind=kind, kv=rng.choice(["e4m3", "int8"]), d=rng.choice([64, 128]), G=1, n=1, ragged_counts=False,
             causal=kind != "attend", accumulate=True, tokens_first=rng.random() < 0.5)
    room = 1 << 22  # entries of all heads
    c["hi"] = hi = _spread(rng, 40, 60000)
    c["H"] = H = min(rng.randint(1, 40), max(1, room // hi))
    c["B"] = max(1, min(_spread(rng, 1, 64), room // (hi * H)))
    c["lo"] = rng.randint(0 if kind == "attend" else 1, hi)
    if kind in ("step", "attend"):
        c["G"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c["n"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["accumulate"] = kind == "step" or rng.random() < 0.5
        c["ragged_counts"] = rng.random() < 0.5
    elif kind == "fill":
        c["n"], c["hi"], c["lo"] = hi, min(hi, 500), min(c["lo"], 500, hi)
        c["ragged_counts"] = rng.random() < 0.5
    else:
        budget = max(2, int(hi * rng.uniform(0.05, 0.6)))
        c["k_local"] = rng.randint(0, budget)
        c["k_heavy"] = budget - c["k_local"]
        c["n_sink"] = rng.choice([0, min(4, c["k_heavy"])])
        c["score_mode"] = rng.choice([0, 1])
    return c


def _lengths(c):
    """Entries of each sequence before the call: spread over lo .. hi."""
    return [c["lo"] + (c["hi"] - c["lo"]) * ((37 * b + 100) % 101) // 100 for b in range(c["B"])]


def _counts(c):
    """New tokens (or queries) of each sequence."""
    if not c["ragged_counts"]:
        return [c["n"]] * c["B"]
    return [c["n"] - (29 * b) % (c["n"] + (c["kind"] == "fill")) for b in range(c["B"])]


def _appends(c):
    return c["kind"] in ("step", "fill")


def work(c):
    lens, counts, d, H, G = _lengths(c), _counts(c), c["d"], c["H"], c["G"]
    new = sum(counts)
    entry = 2 * d + 8 / BLOCK  # codes and scales of one entry
    if c["kind"] == "fill":
        return {"bytes": H * new * (4 * d + entry + 8), "flops": 0}
    if c["kind"] == "evict":
        k = c["k_heavy"] + c["k_local"]
        cut = [n for n in lens if n > k]
        return {"bytes": H * sum(4 * n + k * (2 * entry + 16) for n in cut) + 4 * len(lens), "flops": 0}
    total = [a + (b if _appends(c) else 0) for a, b in zip(lens, counts)]
    rows = H * G * new
    moved = H * sum(total) * (entry + (8 if c["accumulate"] else 0)) + rows * (4 * d + 4)
    if _appends(c):
        moved += H * new * (4 * d + 8)
    return {"bytes": moved, "flops": 4 * d * H * G * sum(a * b for a, b in zip(total, counts))}


# ------------------------------------------------------------ the plain forms

def _scale_of(amax, kv):
    """The least power of two, 2^-100 at least, that brings amax to the largest code."""
    m, e = torch.frexp(amax)
    lm, le = math.frexp(LIMIT[kv])
    e = torch.where(m <= lm, e - le, e - le + 1)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(x, kv):
    if kv == "int8":
        return torch.round(x).to(torch.int8)
    return x.to(torch.float8_e4m3fn)


def _take(t, at):
    """Rows `at` [B, W] of each head of t [B, H, N, ...]."""
    B, H = t.shape[:2]
    bytes_ = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    b = torch.arange(B, device=t.device)[:, None, None]
    h = torch.arange(H, device=t.device)[None, :, None]
    got = bytes_[b, h, at[:, None, :]]
    return got.view(t.dtype) if t.dtype == torch.float8_e4m3fn else got


def _put(t, at, ok, value):
    """The opposite of _take, where `ok` [B, W] (or with heads, [B, H, W])."""
    B, H = t.shape[:2]
    if t.dtype == torch.float8_e4m3fn:
        t, value = t.view(torch.uint8), value.view(torch.uint8)
    ok = (ok if ok.dim() == 3 else ok[:, None, :]).expand(B, H, at.shape[-1])
    b, h, w = ok.nonzero(as_tuple=True)
    t[b, h, at[b, w]] = value[b, h, w]


def _append_rows(codes, scale, x, lens, counts, kv):
    """x [B, H, n, d] quantised behind the first `lens` rows of codes [B, H, cap, d]."""
    B, H, cap, d = codes.shape
    n = x.shape[2]
    dev = x.device
    first = lens // BLOCK
    blocks = first[:, None] + torch.arange((n + BLOCK - 1) // BLOCK + 1, device=dev)   # every block that may change
    at = (blocks[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(1)     # and its entries
    old = at < lens[:, None]
    new = (at >= lens[:, None]) & (at < (lens + counts)[:, None])
    held = (old | new) & (at < cap)
    at = at.clamp(max=cap - 1)
    from_x = (at - lens[:, None]).clamp(0, n - 1)
    xs = _take(x.float(), from_x) * new[:, None, :, None]
    amax = xs.abs().amax(-1).unflatten(2, (-1, BLOCK)).amax(-1)                         # [B, H, blocks]
    touched = new.unflatten(1, (-1, BLOCK)).any(-1)
    blocks = blocks.clamp(max=scale.shape[2] - 1)
    before = torch.where(old.unflatten(1, (-1, BLOCK)).any(-1)[:, None], _take(scale, blocks), 0.0)
    after = torch.maximum(before, _scale_of(amax, kv))
    s1 = after.repeat_interleave(BLOCK, 2)[..., None]
    s0 = before.repeat_interleave(BLOCK, 2)[..., None]
    value = torch.where(old[:, None, :, None], _take(codes, at).float() * (s0 / s1), xs / s1)
    _put(codes, at, held & touched.repeat_interleave(BLOCK, 1), _codes(value, kv))
    _put(scale, blocks, touched, after)


def _append(s):
    c = s["case"]
    for codes, scale, x in ((s["K"], s["K_scale"], s["k"]), (s["V"], s["V_scale"], s["v"])):
        _append_rows(codes, scale, x, s["lengths"], s["counts"], c["kv"])
    n = s["k"].shape[2]
    i = torch.arange(n, device=s["k"].device)
    at, ok = s["lengths"][:, None] + i, i < s["counts"][:, None]
    at = at.clamp(max=s["pos"].shape[2] - 1)
    B, H = s["pos"].shape[:2]
    where = (s["position"][:, None] + i).to(torch.int32)[:, None, :].expand(B, H, n)
    _put(s["pos"], at, ok, where)
    _put(s["score"], at, ok, s["first_score"] if "first_score" in s else torch.zeros_like(s["score"][:, :, :1]).expand(B, H, n))


def _values(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK, 2)[..., None]


def _attend(s, total):
    c = s["case"]
    B, H, G, n, d = c["B"], c["H"], c["G"], c["n"], c["d"]
    cap = s["K"].shape[2]
    dev = s["q"].device
    q = s["q"].float().reshape(B, H, G * n, d)
    logits = (q @ _values(s["K"], s["K_scale"]).transpose(2, 3)).mul_(d ** -0.5).view(B, H, G, n, cap)
    i = torch.arange(n, device=dev)
    end = (total - s["counts"])[:, None] + i + 1 if c["causal"] else total[:, None].expand(B, n)
    live = i < s["counts"][:, None]                                                     # [B, n]
    seen = (torch.arange(cap, device=dev) < end[..., None]) & live[..., None]           # [B, n, cap]
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    w = logits.sub_(top).exp_()
    mass = w.sum(-1, keepdim=True)
    w = w.div_(torch.where(mass > 0, mass, 1.0))
    out = (w.view(B, H, G * n, cap) @ _values(s["V"], s["V_scale"])).view(B, H * G, n, d)
    lse = (mass.log() + top).view(B, H * G, n)
    s["out"].copy_(torch.where(live[:, None, :, None], out.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(live[:, None, :], lse, s["lse"]))
    if c["accumulate"]:
        s["score"] += w.sum((2, 3))


def _evict(s):
    c = s["case"]
    lens, k, kl = s["lengths"], c["k_heavy"] + c["k_local"], c["k_local"]
    B, H, cap = s["score"].shape
    i = torch.arange(cap, device=lens.device)
    key = s["score"]
    if c["score_mode"]:
        key = key / (s["position"][:, None, None] - s["pos"]).clamp(min=1).float()
    safe = (i >= (lens - kl)[:, None])[:, None] | (s["pos"] < c["n_sink"])
    key = torch.where(safe, math.inf, key)
    order = key.sort(dim=-1, stable=True).indices
    gone = (i < (lens - k)[:, None])[:, None].expand(B, H, cap)
    dropped = torch.zeros_like(key, dtype=torch.bool).scatter_(2, order, gone)
    kept = ~dropped & (i < lens[:, None])[:, None]
    slot = kept.cumsum(-1) - 1
    cut = lens > k
    last = k if k < cap else cap
    b, h, j = (kept & cut[:, None, None]).nonzero(as_tuple=True)
    src = torch.zeros(B, H, last, dtype=torch.long, device=lens.device)
    src[b, h, slot[b, h, j]] = j
    b, h = torch.arange(B, device=lens.device)[:, None, None], torch.arange(H, device=lens.device)[None, :, None]
    pad = -last % BLOCK
    for codes, scale in ((s["K"], s["K_scale"]), (s["V"], s["V_scale"])):
        rows = codes.view(torch.uint8)[b, h, src].view(codes.dtype).float() * scale[b, h, src // BLOCK][..., None]
        rows = torch.nn.functional.pad(rows, (0, 0, 0, pad)).unflatten(2, (-1, BLOCK))
        fresh = _scale_of(rows.abs().amax((-1, -2)), c["kv"])
        new = _codes(rows / fresh[..., None, None], c["kv"]).flatten(2, 3)[:, :, :last]
        codes.view(torch.uint8)[cut, :, :last] = new.view(torch.uint8)[cut]
        scale[:, :, : fresh.shape[2]] = torch.where(cut[:, None, None], fresh, scale[:, :, : fresh.shape[2]])
    for t in (s["pos"], s["score"]):
        t[:, :, :last] = torch.where(cut[:, None, None], t[b, h, src], t[:, :, :last])
    return lens.clamp(max=k).to(torch.int32)


# ------------------------------------------------------------ inputs and runs

def prepare(case, seed):
    """A cache as it is in use: keys with a shared direction of power-law strength, queries along it, scores that fell
    with age; the places behind each sequence's last entry hold what earlier sequences left."""
    c, dev = case, "cuda"
    B, H, G, n, d = c["B"], c["H"], c["G"], c["n"], c["d"]
    g = torch.Generator(dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev).clamp_(min=1e-6)

    u = torch.nn.functional.normalize(normal(B, H, 1, d), dim=-1)

    def keys(m):
        return normal(B, H, m, d).addcmul_(uniform(B, H, m, 1).pow_(-1 / 1.5).clamp_(max=8), u)

    def layout(x):
        """Rows as the path has them: [B, heads, n, d], or the same as a view of token-first rows."""
        x = x.to(torch.bfloat16)
        return x.transpose(1, 2).contiguous().transpose(1, 2) if c["tokens_first"] else x

    lens, counts = _lengths(c), _counts(c)
    most = max(a + (b if _appends(c) else 0) for a, b in zip(lens, counts))
    cap = max(BLOCK, -(-most // BLOCK) * BLOCK)
    s = {"case": c}
    for name in ("K", "V"):
        if c["kind"] == "fill" and max(lens) == 0:  # a cache just made
            s[name] = torch.zeros(B, H, cap, d, device=dev).to(STORE[c["kv"]])
            s[name + "_scale"] = torch.zeros(B, H, cap // BLOCK, device=dev)
            continue
        x = (keys(cap) if name == "K" else normal(B, H, cap, d)).to(torch.bfloat16).unflatten(2, (-1, BLOCK))
        s[name + "_scale"] = _scale_of(x.abs().amax((-1, -2)).float(), c["kv"])
        s[name] = _codes(x.float().div_(s[name + "_scale"][..., None, None]), c["kv"]).flatten(2, 3)
    gaps = (uniform(B, H, cap) < 0.3).int() + 1  # positions that were kept so far
    s["pos"] = (gaps.cumsum(-1) - gaps[..., :1]).int() if c["kind"] == "evict" else torch.arange(cap, device=dev, dtype=torch.int32).expand(B, H, cap).contiguous()
    age = torch.arange(cap, 0, -1, device=dev).float()
    s["score"] = uniform(B, H, cap).pow_(4).mul_(age).mul_(G / 8)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    s["position"] = s["pos"][:, :, max(lens) - 1].amax(-1) + 1 if c["kind"] == "evict" else s["lengths"].clone()
    if _appends(c):
        s["k"], s["v"] = layout(keys(n)), layout(normal(B, H, n, d))
    if c["kind"] == "fill":
        s["first_score"] = uniform(B, H, n).mul_(4)
    if c["kind"] in ("step", "attend"):
        s["q"] = layout((normal(B, H, G, n, d) + 2 * u[:, :, :, None]).flatten(1, 2))
        s["out"] = torch.zeros(B, H * G, n, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(B, H * G, n, device=dev)
    if own:
        from h2o_heavy_hitter_decode_gb300 import H2OBlockCache
        cache = H2OBlockCache(B, H, d, cap, group=G, max_queries=n if c["kind"] in ("step", "attend") else 1, kv=c["kv"])
        for name in ("K", "V", "K_scale", "V_scale", "pos", "score"):
            getattr(cache, name).copy_(s[name])
            s[name] = getattr(cache, name)
        s["cache"] = cache
        if not c["ragged_counts"]:
            s["counts"] = None
    return s


def _state(s):
    return {n: s[n] for n in ("K", "V", "K_scale", "V_scale", "pos", "score")}


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        cache = s["cache"]
        if kind == "fill":
            cache.append(s["k"], s["v"], s["lengths"], s["counts"], position=s["position"], score=s["first_score"])
            return _state(s)
        if kind == "step":
            cache.step(s["q"], s["k"], s["v"], s["lengths"], s["counts"], position=s["position"],
                       accumulate=c["accumulate"], out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"], **_state(s)}
        if kind == "attend":
            cache.attend(s["q"], s["lengths"], s["counts"], causal=c["causal"], accumulate=c["accumulate"],
                         out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"], "score": s["score"]}
        lengths = cache.evict(s["lengths"], c["k_heavy"], c["k_local"], n_sink=c["n_sink"], score_mode=c["score_mode"],
                              position=s["position"])
        return {"lengths": lengths, **_state(s)}
    if kind == "fill":
        _append(s)
        return _state(s)
    if kind == "step":
        _append(s)
        _attend(s, s["lengths"] + s["counts"])
        return {"out": s["out"], "lse": s["lse"], **_state(s)}
    if kind == "attend":
        _attend(s, s["lengths"])
        return {"out": s["out"], "lse": s["lse"], "score": s["score"]}
    return {"lengths": _evict(s), **_state(s)}


# --------------------------------------------- the definitions, in 64 bits

def _round_code(x, kv):
    """x (64 bits, at most the largest code) to the nearest code, ties to even."""
    if kv == "int8":
        return torch.round(x)
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)  # spacing of e4m3 numbers at x: 3 bits after the leading one
    return torch.round(x / step) * step


def _power(amax, kv):
    """The scale of values up to amax (64 bits)."""
    e = torch.ceil(torch.log2(amax / LIMIT[kv]))
    e = torch.where(amax <= LIMIT[kv] * torch.exp2(e - 1), e - 1, torch.where(amax > LIMIT[kv] * torch.exp2(e), e + 1, e))
    return torch.exp2(torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP))


def _exact_append(codes, scale, x, a, b, kv):
    """x [H, b - a, d] into rows a .. b-1 of codes [H, cap, d], block by block where a block has rows already."""
    whole = min(b, -(-a // BLOCK) * BLOCK)   # rows a .. whole-1 end a block that holds entries
    if whole > a:
        j = a // BLOCK
        new = x[:, : whole - a]
        s1 = torch.maximum(scale[:, j], _power(new.abs().amax((1, 2)), kv))
        rows = codes[:, j * BLOCK : a] * (scale[:, j] / s1)[:, None, None]
        codes[:, j * BLOCK : a] = _round_code(rows, kv)
        codes[:, a:whole] = _round_code(new / s1[:, None, None], kv)
        scale[:, j] = s1
    if b > whole:
        rest = x[:, whole - a :]
        full = torch.nn.functional.pad(rest, (0, 0, 0, -rest.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))
        s1 = _power(full.abs().amax((-1, -2)), kv)
        codes[:, whole:b] = _round_code(full / s1[..., None, None], kv).flatten(1, 2)[:, : b - whole]
        j = whole // BLOCK
        scale[:, j : j + s1.shape[1]] = s1


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    lens, counts = _lengths(c), _counts(c)
    B, H, G, d, kv = c["B"], c["H"], c["G"], c["d"], c["kv"]
    keep = {n: torch.empty_like(s[n], dtype=torch.float64) for n in ("K", "V", "K_scale", "V_scale", "score")}
    if "out" in s:
        keep["out"], keep["lse"] = torch.zeros_like(s["out"], dtype=torch.float64), s["lse"].double()
    for b in range(B):
        t = {n: s[n][b].double() for n in ("K", "V", "K_scale", "V_scale", "score")}
        total = lens[b]
        if _appends(c):
            total += counts[b]
            if counts[b]:
                for n in ("K", "V"):
                    _exact_append(t[n], t[n + "_scale"], s[n.lower()][b, :, : counts[b]].double(), lens[b], total, kv)
                t["score"][:, lens[b] : total] = s["first_score"][b, :, : counts[b]].double() if c["kind"] == "fill" else 0
        if "out" in s and counts[b] and total:
            keys = (t["K"] * t["K_scale"].repeat_interleave(BLOCK, 1)[..., None])[:, :total]
            values = (t["V"] * t["V_scale"].repeat_interleave(BLOCK, 1)[..., None])[:, :total]
            q = s["q"][b, :, : counts[b]].double().unflatten(0, (H, G))
            logits = torch.einsum("hgid,hjd->hgij", q, keys) / math.sqrt(d)
            if c["causal"]:
                hidden = torch.ones(counts[b], total, dtype=torch.bool, device=q.device).triu(total - counts[b] + 1)
                logits[..., hidden] = -math.inf
            keep["lse"][b, :, : counts[b]] = torch.logsumexp(logits, -1).flatten(0, 1)
            w = torch.softmax(logits, -1)
            keep["out"][b, :, : counts[b]] = torch.einsum("hgij,hjd->hgid", w, values).flatten(0, 1)
            if c["accumulate"]:
                t["score"][:, :total] += w.sum((1, 2))
        elif "out" in s:
            keep["lse"][b, :, : counts[b]] = -math.inf
        k = c.get("k_heavy", 0) + c.get("k_local", 0)
        if c["kind"] == "evict" and total > k:
            first = total - c["k_local"]
            key = t["score"][:, :first]
            if c["score_mode"]:
                key = (key / (s["position"][b] - s["pos"][b, :, :first]).clamp(min=1)).float().double()
            key = torch.where(s["pos"][b, :, :first] < c["n_sink"], math.inf, key)
            best = key.flip(-1).sort(dim=-1, descending=True, stable=True).indices[:, : c["k_heavy"]]  # later ones first
            mine = torch.cat([first - 1 - best, torch.arange(first, total, device=best.device).expand(H, -1)], 1).sort(-1).values
            h = torch.arange(H, device=best.device)[:, None]
            t["score"][:, :k] = t["score"][h, mine].clone()
            for n in ("K", "V"):
                rows = t[n][h, mine] * t[n + "_scale"][h, mine // BLOCK][..., None]
                _exact_append(t[n], t[n + "_scale"], rows, 0, k, kv)
        for n, x in t.items():
            keep[n][b] = x
    if kv == "int8":  # whole numbers: compared with the plain form's
        keep["K"] = keep["V"] = None
    if c["kind"] == "attend":
        return {n: keep[n] for n in ("out", "lse", "score")}
    keep["pos"] = None
    if c["kind"] == "evict":
        keep["lengths"] = None
    return keep
