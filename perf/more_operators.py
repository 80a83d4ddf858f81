"""Cases for the operators around a block-scaled 8-bit K/V cache (``H2OBlockCache``).

  rotate   queries and keys normed per head and rotated by their positions, before they meet the cache (``H2ORotary``)
  sparse   decode over a long cache: per query token and cached head the blocks of 32 entries with the highest bound on
           their logits are chosen, attended to and scored; with the append of the new tokens, or alone
  copy     sequences of a cache forked, reordered, compacted, in place or out of another cache

``run`` computes them in elementary torch operations, or with the framework's
calls where ``own`` is set; ``exact`` computes them in 64 bits from the
definitions."""
import math

import torch

own = False

BLOCK = 32                               # entries that share a scale
LIMIT = {"e4m3": 448.0, "int8": 127.0}   # largest code
UNIT = {"e4m3": 4.0, "int8": 1.0}        # what 1 of a block's bounds stands for, in codes
STORE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
MIN_EXP = -100                           # smallest scale: 2^-100


def listed():
    rot = dict(kind="rotate", dtype="bf16", d=128, dims=128, axes=1, interleaved=False, norm=True, far=8192,
               ragged_counts=False, tokens_first=True)
    sp = dict(kind="sparse", kv="e4m3", d=128, G=1, n=1, n_first=1, n_last=2, ragged_counts=False, appends=True,
              causal=True, accumulate=True, tokens_first=False)
    cp = dict(kind="copy", kv="e4m3", d=128, bounds=True, rows_from=0)
    return [
        # one token of one sequence: latency
        dict(rot, name="rotate one token", B=1, H=32, G=1, n=1),
        # a decode step of a batch far into a long stream, grouped queries
        dict(rot, name="rotate batch", B=64, H=8, G=8, n=1, far=4194304),
        # 8K-token prompts
        dict(rot, name="rotate prompts", B=16, H=32, G=1, n=8192),
        # patches of images and video on three axes, an odd number, half of the dimensions rotated in neighbouring pairs
        dict(rot, name="rotate patches", B=3, H=16, G=1, n=2257, d=64, dims=32, axes=3, interleaved=True, norm=False,
             ragged_counts=True, dtype="fp32", tokens_first=False),
        # one sequence of an OPT-6.7B-shaped layer, its whole text cached: latency
        dict(sp, name="sparse one sequence", B=1, H=32, lo=2559, hi=2559, n_blocks=16),
        # sequences of every age, four query heads share a cached one
        dict(sp, name="sparse groups of 4", kv="int8", B=16, H=8, G=4, lo=3001, hi=8447, n_blocks=64, tokens_first=True),
        # draft tokens verified, each with its own choice
        dict(sp, name="sparse draft tokens", B=8, H=8, G=8, n=5, d=64, lo=1000, hi=8100, n_blocks=40,
             ragged_counts=True, tokens_first=True),
        # one long text, groups of eight
        dict(sp, name="sparse long", B=1, H=8, G=8, lo=262000, hi=262000, n_blocks=128),
        # a batch of long texts
        dict(sp, name="sparse long batch", B=16, H=8, G=8, lo=20000, hi=65500, n_blocks=128),
        # four beams over one short text
        dict(cp, name="copy beams", pattern="beams", B=4, H=32, lo=255, hi=255),
        # a batch of beams of an OPT-30B-shaped layer
        dict(cp, name="copy batch", pattern="beams", kv="int8", B=64, H=56, lo=700, hi=2047, bounds=False),
        # two prompts of 8K tokens forked into the rows of a running batch
        dict(cp, name="copy fork", pattern="fork", B=16, H=32, lo=8001, hi=8192, rows_from=2),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "sparse", "sparse", "sparse", "copy", "copy"])
    c = dict(kind=kind, d=rng.choice([64, 128]))
    if kind == "rotate":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        c["H"], c["G"] = rng.randint(1, 40), rng.choice([1, 1, 2, 4, 5, 8])
        tokens = max(1, _spread(rng, 1, 4000000) // (c["H"] * (c["G"] + 1)))
        c["n"] = min(tokens, _spread(rng, 1, 8192))
        c["B"] = max(1, min(64, tokens // c["n"]))
        c["dims"] = 16 * rng.randint(1, c["d"] // 16)
        c["axes"] = rng.choice([1, 1, 2, 3, 4])
        c["interleaved"] = rng.random() < 0.4
        c["norm"] = rng.random() < 0.6
        c["far"] = _spread(rng, 1, 1 << 30)
        c["ragged_counts"] = rng.random() < 0.4
        c["tokens_first"] = rng.random() < 0.5
        return c
    c["kv"] = rng.choice(["e4m3", "int8"])
    room = 1 << 22  # entries of all heads
    if kind == "sparse":
        c["hi"] = hi = _spread(rng, 40, 100000)
        c["H"] = H = min(rng.randint(1, 40), max(1, room // hi))
        c["B"] = max(1, min(_spread(rng, 1, 64), room // (hi * H)))
        c["appends"] = rng.random() < 0.7
        c["causal"] = c["appends"] or rng.random() < 0.5
        c["lo"] = rng.randint(0 if not c["appends"] else 1, hi)
        c["n"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["G"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        c["n_first"], c["n_last"] = rng.choice([0, 1, 1, 2]), rng.choice([1, 2, 2, 5])
        c["n_blocks"] = c["n_first"] + c["n_last"] + _spread(rng, 1, 200) - rng.choice([0, 1])
        # what a step attends to stays below the largest listed one
        c["B"] = max(1, min(c["B"], 16384 // (H * c["n"] * min(c["n_blocks"], -(-hi // BLOCK)))))
        c["accumulate"] = c["appends"] or rng.random() < 0.5
        c["ragged_counts"] = rng.random() < 0.5
        c["tokens_first"] = rng.random() < 0.5
        return c
    c["pattern"] = rng.choice(["beams", "cycle", "compact", "fork"])
    c["hi"] = hi = _spread(rng, 20, 60000)
    c["H"] = H = min(rng.randint(1, 40), max(1, room // (2 * hi)))
    c["B"] = max(2, min(_spread(rng, 2, 100), room // (hi * H)))
    c["lo"] = rng.randint(0, hi)
    c["bounds"] = rng.random() < 0.5
    c["rows_from"] = rng.randint(1, 5) if c["pattern"] == "fork" else 0
    return c


def _lengths(c, rows=None):
    """Entries of each sequence before the call: spread over lo .. hi."""
    return [c["lo"] + (c["hi"] - c["lo"]) * ((37 * b + 100) % 101) // 100 for b in range(rows or c["B"])]


def _counts(c):
    """New tokens (or queries) of each sequence."""
    if not c["ragged_counts"]:
        return [c["n"]] * c["B"]
    return [c["n"] - (29 * b) % c["n"] for b in range(c["B"])]


def _axis(c):
    """The axis of each pair of dimensions: runs of nearly equal length, as the models have them."""
    pairs = c["dims"] // 2
    return [i * c["axes"] // pairs for i in range(pairs)]


def _parents(c):
    """The row whose content each row of the cache receives; -1: it stays."""
    B = c["B"]
    if c["pattern"] == "beams":  # beams of four: the better ones go on twice
        return [min(B - 1, b - b % 4 + (0, 0, 1, 3)[(b + b // 4) % 4]) for b in range(B)]
    if c["pattern"] == "cycle":
        return [(b + 1) % B for b in range(B)]
    if c["pattern"] == "compact":  # finished sequences leave, the others move up
        live = [b for b in range(B) if (7 * b + 1) % 4]
        return live + [-1] * (B - len(live))
    return [-1 if b % 5 == 4 else b * c["rows_from"] // B for b in range(B)]


def work(c):
    d, H = c["d"], c["H"]
    if c["kind"] == "rotate":
        rows = sum(_counts(c)) * H * (c["G"] + 1)
        size = TYPES[c["dtype"]].itemsize
        return {"bytes": 2 * rows * d * size + 4 * c["axes"] * c["B"] * c["n"], "flops": rows * (3 * c["dims"] + (3 * d if c["norm"] else 0))}
    entry = 2 * d + 8 / BLOCK  # codes and scales of one entry
    if c["kind"] == "copy":
        lens, parents = _lengths(c, c["rows_from"] or None), _parents(c)
        moved = [p for b, p in enumerate(parents) if p >= 0 and (c["rows_from"] or p != b)]
        blocks = [-(-n // BLOCK) for n in lens]
        total = sum(blocks[p] for p in set(moved)) + sum(blocks[p] for p in moved)
        return {"bytes": H * total * (BLOCK * (entry + 8) + (2 * d if c["bounds"] else 0)) + 12 * c["B"], "flops": 0}
    lens, counts, G = _lengths(c), _counts(c), c["G"]
    moved = flops = 0
    for a, b in zip(lens, counts):
        total = a + (b if c["appends"] else 0)
        blocks = -(-total // BLOCK)
        chosen = min(blocks, c["n_blocks"])
        rest = blocks - c["n_first"] - c["n_last"] if blocks > c["n_blocks"] else 0
        seen = min(total, chosen * BLOCK)
        moved += rest * (2 * d + 4) + seen * (entry + (8 if c["accumulate"] else 0)) + b * G * (4 * d + 4) + b * 4 * c["n_blocks"]
        moved += b * (4 * d + entry + 8) if c["appends"] else 0
        flops += b * G * (4 * d * seen + 4 * d * rest)
    return {"bytes": H * moved, "flops": H * flops}


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


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _take(t, at):
    """Entries `at` [B, W] of each head of t [B, H, N, ...]."""
    B, H = t.shape[:2]
    b = torch.arange(B, device=t.device)[:, None, None]
    h = torch.arange(H, device=t.device)[None, :, None]
    got = _bytes(t)[b, h, at[:, None, :]]
    return got.view(t.dtype) if t.dtype == torch.float8_e4m3fn else got


def _put(t, at, ok, value):
    """The opposite of _take, where `ok` [B, W]."""
    b, h, w = ok[:, None, :].expand(-1, t.shape[1], -1).nonzero(as_tuple=True)
    _bytes(t)[b, h, at[b, w]] = _bytes(value)[b, h, w]


def _bounds(codes, kv):
    """Least and largest code of each dimension of blocks [..., 32, d], as whole numbers of units: [..., 2, d]."""
    x = codes.float()
    return torch.stack([(x.amin(-2) / UNIT[kv]).floor(), (x.amax(-2) / UNIT[kv]).ceil()], -2).to(torch.int8)


def _append(s):
    """The new rows quantised behind each sequence's entries; the bounds of the blocks that they touch."""
    c = s["case"]
    lens, counts, n, kv = s["lengths"], s["counts"], c["n"], c["kv"]
    dev, cap = lens.device, s["K"].shape[2]
    blocks = (lens // BLOCK)[:, None] + torch.arange((n + BLOCK - 1) // BLOCK + 1, device=dev)
    at = (blocks[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(1)
    old, new = at < lens[:, None], (at >= lens[:, None]) & (at < (lens + counts)[:, None])
    in_block = lambda x: x.unflatten(1, (-1, BLOCK)).any(-1)  # noqa: E731
    touched = in_block(new)
    held = (old | new) & touched.repeat_interleave(BLOCK, 1)
    at, blocks = at.clamp(max=cap - 1), blocks.clamp(max=cap // BLOCK - 1)
    from_x = (at - lens[:, None]).clamp(0, n - 1)
    for name in ("K", "V"):
        codes, scale, x = s[name], s[name + "_scale"], s[name.lower()]
        xs = _take(x.float(), from_x) * new[:, None, :, None]
        amax = xs.abs().amax(-1).unflatten(2, (-1, BLOCK)).amax(-1)
        before = torch.where(in_block(old)[:, None], _take(scale, blocks), 0.0)
        after = torch.maximum(before, _scale_of(amax, kv))
        s1 = after.repeat_interleave(BLOCK, 2)[..., None]
        s0 = before.repeat_interleave(BLOCK, 2)[..., None]
        value = torch.where(old[:, None, :, None], _take(codes, at).float() * (s0 / s1), xs / s1)
        _put(codes, at, held, _codes(value, kv))
        _put(scale, blocks, touched, after)
    rows = _take(s["K"], at).float()
    least = torch.where(held[:, None, :, None], rows, math.inf).unflatten(2, (-1, BLOCK)).amin(-2)
    most = torch.where(held[:, None, :, None], rows, -math.inf).unflatten(2, (-1, BLOCK)).amax(-2)
    fresh = torch.stack([(least / UNIT[kv]).floor(), (most / UNIT[kv]).ceil()], -2)
    _put(s["bounds"], blocks, touched, fresh.clamp(-128, 127).to(torch.int8))
    i = torch.arange(n, device=dev)
    at, ok = (lens[:, None] + i).clamp(max=cap - 1), i < counts[:, None]
    B, H = s["pos"].shape[:2]
    _put(s["pos"], at, ok, (lens[:, None] + i).to(torch.int32)[:, None, :].expand(B, H, n))
    _put(s["score"], at, ok, torch.zeros(B, H, n, device=dev))


def _sparse(s):
    c = s["case"]
    B, H, G, n, d, S = c["B"], c["H"], c["G"], c["n"], c["d"], c["n_blocks"]
    dev, nblk = s["q"].device, s["bounds"].shape[2]
    total = s["lengths"] + (s["counts"] if c["appends"] else 0)
    i = torch.arange(n, device=dev)
    live = i < s["counts"][:, None]                                                       # [B, n]
    end = (total - s["counts"])[:, None] + i + 1 if c["causal"] else total[:, None].expand(B, n)
    last = (end + BLOCK - 1) // BLOCK                                                     # blocks a token sees
    q = s["q"].float().view(B, H, G, n, d).permute(0, 1, 3, 2, 4)                         # [B, H, n, G, d]
    # the bound on a block's logits, from queries in 8 bits: whole numbers below 2^24, exact in any order
    x = torch.round(q / _scale_of(q.abs().amax((-1, -2), keepdim=True), "int8"))
    bound = x.clamp(min=0).flatten(2, 3) @ s["bounds"][:, :, :, 1].float().transpose(2, 3)
    bound += x.clamp(max=0).flatten(2, 3) @ s["bounds"][:, :, :, 0].float().transpose(2, 3)
    key = bound.view(B, H, n, G, nblk).amax(3) * s["K_scale"][:, :, None]
    j = torch.arange(nblk, device=dev)
    sure = (j < c["n_first"]) | (j >= (last - c["n_last"])[..., None])                    # [B, n, nblk]
    key = key.masked_fill(sure[:, None], math.inf).masked_fill((j >= last[..., None])[:, None], -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :S]
    none = (best >= last[:, None, :, None]) | ~live[:, None, :, None]
    best = best.masked_fill(none, nblk).sort(-1).values
    none = best == nblk
    s["blocks"][..., : best.shape[-1]] = torch.where(live[:, None, :, None], best.masked_fill(none, -1).int(), s["blocks"][..., : best.shape[-1]])
    # attention over the entries of the chosen blocks
    at = (best.masked_fill(none, 0)[..., None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(-2)  # [B, H, n, E]
    seen = ~none.repeat_interleave(BLOCK, -1) & (at < end[:, None, :, None])
    b, h = torch.arange(B, device=dev)[:, None, None, None], torch.arange(H, device=dev)[None, :, None, None]
    values = lambda name: (_bytes(s[name])[b, h, at].view(s[name].dtype).float() * s[name + "_scale"][b, h, at // BLOCK][..., None])  # noqa: E731
    logits = (q @ values("K").transpose(-1, -2)).mul_(d ** -0.5)                          # [B, H, n, G, E]
    logits.masked_fill_(~seen[:, :, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    w = logits.sub_(top).exp_()
    mass = w.sum(-1, keepdim=True)
    w = w.div_(torch.where(mass > 0, mass, 1.0))
    out = (w @ values("V")).permute(0, 1, 3, 2, 4).reshape(B, H * G, n, d)
    lse = (mass.log() + top).permute(0, 1, 3, 2, 4).reshape(B, H * G, n)
    s["out"].copy_(torch.where(live[:, None, :, None], out.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(live[:, None, :], lse, s["lse"]))
    if c["accumulate"]:
        s["score"].scatter_add_(2, at.flatten(2), w.sum(3).flatten(2))


def _rotate(s):
    c = s["case"]
    n, r = c["n"], c["dims"]
    i = torch.arange(n, device=s["position"].device)
    position = s["position"] if s["position"].dim() == 3 else (s["position"][:, None] + i)[None]
    angle = position.double()[s["axis"]].permute(1, 2, 0) * s["frequency"]                # [B, n, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    live = (i < s["counts"][:, None])[:, None, :, None]
    for name in ("q", "k"):
        x = s[name].float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"].float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., : r // 2], x[..., r // 2 : r])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        y = torch.cat([turned, x[..., r:]], -1).to(TYPES[c["dtype"]])
        s[name + "_out"].copy_(torch.where(live, y, s[name + "_out"]))


def _copy(s):
    parent = s["parent"].long()
    moves, p = parent >= 0, parent.clamp(min=0)
    most = s["blocks"]
    take = moves[:, None] & (torch.arange(most, device=p.device) < ((s["from_lengths"] + BLOCK - 1) // BLOCK)[p][:, None])
    for name, x in s["from"].items():
        m = most * (BLOCK if name in ("K", "V", "pos", "score") else 1)
        ok = take.repeat_interleave(m // most, 1) if most else take
        to = _bytes(s[name])[:, :, :m]
        ok = ok[:, None].reshape(ok.shape[0], 1, m, *[1] * (to.dim() - 3))
        to.copy_(torch.where(ok, _bytes(x)[:, :, :m][p], to))
    return torch.where(moves, s["from_lengths"][p], s["lengths"])


# ------------------------------------------------------------ inputs and runs

def _cache(c, g, rows, cap, dev):
    """A cache as it is in use: keys with a shared direction of power-law strength, scores that fell with age."""
    H, d = c["H"], c["d"]
    u = torch.nn.functional.normalize(torch.randn(rows, H, 1, d, generator=g, device=dev), dim=-1)
    s = {}
    for name in ("K", "V"):
        x = torch.randn(rows, H, cap, d, generator=g, device=dev)
        if name == "K":
            x.addcmul_(torch.rand(rows, H, cap, 1, generator=g, device=dev).clamp_(min=1e-6).pow_(-1 / 1.5).clamp_(max=8), u)
        x = x.to(torch.bfloat16).unflatten(2, (-1, BLOCK))
        s[name + "_scale"] = _scale_of(x.abs().amax((-1, -2)).float(), c["kv"])
        s[name] = _codes(x.float().div_(s[name + "_scale"][..., None, None]), c["kv"]).flatten(2, 3)
    s["pos"] = torch.arange(cap, device=dev, dtype=torch.int32).expand(rows, H, cap).contiguous()
    age = torch.arange(cap, 0, -1, device=dev).float()
    s["score"] = torch.rand(rows, H, cap, generator=g, device=dev).pow_(4).mul_(age).div_(8)
    if c["kind"] == "sparse" or c["bounds"]:
        s["bounds"] = _bounds(s["K"].unflatten(2, (-1, BLOCK)), c["kv"])
    return s, u


def _held(arrays, c, group=1, n=1):
    """The framework's cache with that content, and its arrays."""
    from h2o_heavy_hitter_decode_gb300 import H2OBlockCache
    B, H, cap, d = arrays["K"].shape
    cache = H2OBlockCache(B, H, d, cap, group=group, max_queries=n, kv=c["kv"], bounds="bounds" in arrays)
    for name, x in arrays.items():
        getattr(cache, name).copy_(x)
    return cache, {name: getattr(cache, name) for name in arrays}


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    B, H, d = c["B"], c["H"], c["d"]

    def layout(x, dtype=torch.bfloat16):
        """Rows as the path has them: [B, heads, n, d], or the same as a view of token-first rows."""
        x = x.to(dtype)
        return x.transpose(1, 2).contiguous().transpose(1, 2) if c["tokens_first"] else x

    if c["kind"] == "rotate":
        G, n, dtype, pairs = c["G"], c["n"], TYPES[c["dtype"]], c["dims"] // 2
        s = {"case": c, "eps": 1e-6, "counts": torch.tensor(_counts(c), dtype=torch.int32, device=dev)}
        for name, heads in (("q", H * G), ("k", H)):
            s[name] = layout(normal(B, heads, n, d), dtype)
            s[name + "_weight"] = normal(d).mul_(0.2).add_(1).to(torch.bfloat16)
            s[name + "_out"] = torch.zeros(B, heads, n, d, dtype=dtype, device=dev)
        s["axis"] = torch.tensor(_axis(c), device=dev)
        s["frequency"] = 10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)
        shape = (B,) if c["axes"] == 1 else (c["axes"], B, n)
        s["position"] = torch.randint(0, c["far"], shape, generator=g, device=dev, dtype=torch.int32)
        if own:
            from h2o_heavy_hitter_decode_gb300 import H2ORotary
            norm = dict(eps=s["eps"], q_weight=s["q_weight"], k_weight=s["k_weight"]) if c["norm"] else {}
            s["rotary"] = H2ORotary(d, frequency=s["frequency"], axis=s["axis"], interleaved=c["interleaved"], **norm)
            if not c["ragged_counts"]:
                s["counts"] = None
        return s

    if c["kind"] == "copy":
        rows, lens = c["rows_from"] or B, _lengths(c, c["rows_from"] or None)
        most = -(-max(lens) // BLOCK)
        cap = max(1, most) * BLOCK
        arrays, _ = _cache(c, g, rows, cap, dev)
        target = arrays
        if c["rows_from"]:  # into a batch that runs already, with room for more
            target, _ = _cache(c, g, B, cap + 4 * BLOCK, dev)
        s = {"case": c, "blocks": most, "from_lengths": torch.tensor(lens, dtype=torch.int32, device=dev)}
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
        s["parent"] = torch.tensor(_parents(c), dtype=torch.int32, device=dev)
        if own:
            s["cache"], target = _held(target, c)
            s["source"], arrays = (_held(arrays, c)[0], None) if c["rows_from"] else (None, None)
        return {**s, **target, "from": arrays}

    G, n = c["G"], c["n"]
    lens, counts = _lengths(c), _counts(c)
    cap = max(1, -(-max(a + (b if c["appends"] else 0) for a, b in zip(lens, counts)) // BLOCK)) * BLOCK
    arrays, u = _cache(c, g, B, cap, dev)
    s = {"case": c, "lengths": torch.tensor(lens, dtype=torch.int32, device=dev),
         "counts": torch.tensor(counts, dtype=torch.int32, device=dev)}
    if c["appends"]:
        s["k"], s["v"] = layout(normal(B, H, n, d) + 2 * u), layout(normal(B, H, n, d))
    s["q"] = layout((normal(B, H, G, n, d) + 2 * u[:, :, :, None]).flatten(1, 2))
    s["out"] = torch.zeros(B, H * G, n, d, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(B, H * G, n, device=dev)
    s["blocks"] = torch.full((B, H, n, c["n_blocks"]), -1, dtype=torch.int32, device=dev)
    if own:
        s["cache"], arrays = _held(arrays, c, G, n)
        if not c["ragged_counts"]:
            s["counts"] = None
    return {**s, **arrays}


def _state(s):
    return {n: s[n] for n in ("K", "V", "K_scale", "V_scale", "pos", "score", "bounds") if n in s}


def run(s):
    c = s["case"]
    if c["kind"] == "rotate":
        if own:
            s["rotary"].apply(s["q"], s["k"], s["position"], s["counts"], q_out=s["q_out"], k_out=s["k_out"])
        else:
            _rotate(s)
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["kind"] == "copy":
        if own:
            lengths = s["cache"].copy(s["parent"], s["lengths"], s["source"], s["from_lengths"] if s["source"] else None)
        else:
            lengths = _copy(s)
        return {"lengths": lengths, **_state(s)}
    if own:
        kept = dict(n_blocks=c["n_blocks"], n_first=c["n_first"], n_last=c["n_last"])
        to = dict(accumulate=c["accumulate"], out=s["out"], lse=s["lse"], blocks=s["blocks"])
        if c["appends"]:
            s["cache"].step_sparse(s["q"], s["k"], s["v"], s["lengths"], counts=s["counts"], **kept, **to)
        else:
            s["cache"].attend_sparse(s["q"], s["lengths"], counts=s["counts"], causal=c["causal"], **kept, **to)
    else:
        if c["appends"]:
            _append(s)
        _sparse(s)
    got = {"out": s["out"], "lse": s["lse"], "blocks": s["blocks"]}
    return {**got, **_state(s)} if c["appends"] else {**got, "score": s["score"]}


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


def _exact_rotate(c, s):
    out = {}
    axis, pairs = _axis(c), c["dims"] // 2
    counts = _counts(c)
    for name in ("q", "k"):
        y = torch.zeros(s[name].shape, dtype=torch.float64, device=s[name].device)
        for b in range(c["B"]):
            x = s[name][b, :, : counts[b]].double()
            if c["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * s[name + "_weight"].double()
            t = torch.arange(counts[b], device=x.device)
            turned = x.clone()
            for i in range(pairs):
                where = s["position"][b] + t if c["axes"] == 1 else s["position"][axis[i], b, : counts[b]]
                angle = where.double() * 10000.0 ** (-i / pairs)
                lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + pairs)
                turned[..., lo] = x[..., lo] * angle.cos() - x[..., hi] * angle.sin()
                turned[..., hi] = x[..., lo] * angle.sin() + x[..., hi] * angle.cos()
            y[b, :, : counts[b]] = turned
        out[name] = y
    return out


def _exact_copy(c, s):
    lens, parents = _lengths(c, c["rows_from"] or None), _parents(c)
    old = {n: x.clone() for n, x in s["from"].items()}
    for b, p in enumerate(parents):
        if p < 0:
            continue
        m = -(-lens[p] // BLOCK)
        for n, x in old.items():
            rows = m * BLOCK if n in ("K", "V", "pos", "score") else m
            _bytes(s[n])[b, :, :rows] = _bytes(x)[p, :, :rows]
    got = {n: s[n].double() for n in ("K", "V", "K_scale", "V_scale", "score")}
    if c["kv"] == "int8":  # whole numbers: compared with the plain form's
        got["K"] = got["V"] = None
    return {**got, "lengths": None, "pos": None, **({"bounds": None} if c["bounds"] else {})}


def _exact_sparse(c, s):
    lens, counts = _lengths(c), _counts(c)
    H, G, d, kv = c["H"], c["G"], c["d"], c["kv"]
    dev = s["q"].device
    keep = {n: s[n].double() for n in ("K", "V", "K_scale", "V_scale", "score")}
    keep["out"], keep["lse"] = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev), s["lse"].double()
    bounds = s["bounds"].long()
    heads = torch.arange(H, device=dev)[:, None]
    for b in range(c["B"]):
        a, total = lens[b], lens[b] + (counts[b] if c["appends"] else 0)
        first = a // BLOCK
        for j in range(first, -(-total // BLOCK) if total > a else first):  # blocks that receive rows
            lo, hi, base = max(a, j * BLOCK), min(total, (j + 1) * BLOCK), j * BLOCK
            for n in ("K", "V"):
                codes, scale = keep[n][b], keep[n + "_scale"][b]
                new = s[n.lower()][b, :, lo - a : hi - a].double()
                s1 = _power(new.abs().amax((1, 2)), kv)
                if a > base:
                    s1 = torch.maximum(s1, scale[:, j])
                    codes[:, base:a] = _round_code(codes[:, base:a] * (scale[:, j] / s1)[:, None, None], kv)
                codes[:, lo:hi] = _round_code(new / s1[:, None, None], kv)
                scale[:, j] = s1
            rows = keep["K"][b][:, base:hi] / UNIT[kv]
            bounds[b, :, j, 0], bounds[b, :, j, 1] = rows.amin(1).floor().long(), rows.amax(1).ceil().long()
        keep["score"][b, :, a:total] = 0
        for t in range(counts[b]):
            end = total - counts[b] + t + 1 if c["causal"] else total
            blocks = -(-end // BLOCK)
            q = s["q"][b, :, t].double().unflatten(0, (H, G))
            if end <= 0:
                keep["lse"][b, :, t] = -math.inf
                continue
            chosen = torch.arange(blocks, device=dev).expand(H, -1)
            if blocks > c["n_blocks"]:
                x = torch.round(q / _power(q.abs().amax((1, 2)), "int8")[:, None, None])
                low, high = bounds[b, :, :blocks, 0].double(), bounds[b, :, :blocks, 1].double()
                m = x.clamp(min=0) @ high.transpose(1, 2) + x.clamp(max=0) @ low.transpose(1, 2)
                key = m.amax(1) * keep["K_scale"][b, :, :blocks]
                mid = key[:, c["n_first"] : blocks - c["n_last"]]
                wanted = c["n_blocks"] - c["n_first"] - c["n_last"]
                best = (-mid).sort(dim=-1, stable=True).indices[:, :wanted] + c["n_first"]
                ends = [*range(c["n_first"]), *range(blocks - c["n_last"], blocks)]
                chosen = torch.cat([best, torch.tensor(ends, device=dev).expand(H, -1)], 1).sort(-1).values
            at = (chosen[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(1)
            unseen = at >= end
            at = at.clamp(max=end - 1)
            keys = keep["K"][b][heads, at] * keep["K_scale"][b][heads, at // BLOCK][..., None]
            values = keep["V"][b][heads, at] * keep["V_scale"][b][heads, at // BLOCK][..., None]
            logits = (q @ keys.transpose(1, 2) / math.sqrt(d)).masked_fill(unseen[:, None], -math.inf)
            w = torch.softmax(logits, -1)
            keep["lse"][b, :, t] = torch.logsumexp(logits, -1).flatten()
            keep["out"][b, :, t] = (w @ values).flatten(0, 1)
            if c["accumulate"]:
                keep["score"][b].scatter_add_(1, at, w.sum(1))
    if not c["appends"]:
        return {n: keep[n] for n in ("out", "lse", "score")} | {"blocks": None}
    if kv == "int8":  # whole numbers: compared with the plain form's
        keep["K"] = keep["V"] = None
    return {**keep, "blocks": None, "pos": None, "bounds": None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotate":
        return _exact_rotate(case, s)
    if case["kind"] == "copy":
        return _exact_copy(case, s)
    return _exact_sparse(case, s)
