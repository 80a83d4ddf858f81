"""A plain 64-bit implementation of the block-scaled 8-bit cache on the CPU,
one sequence and head at a time, and the tolerances of the GPU kernels."""
from __future__ import annotations

import math

import torch

BLOCK = 32
LIMIT = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -100


def pow2_scale(amax: float, kv: str) -> float:
    """Least 2^e, e >= -100, with amax <= LIMIT * 2^e."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.frexp(amax)[1] - 12)
        while amax > LIMIT[kv] * 2.0 ** e:
            e += 1
    return 2.0 ** e


def round_code(x: torch.Tensor, kv: str) -> torch.Tensor:
    """float64 values to codes (as float64), nearest, ties to even, saturating."""
    if kv == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


class RefCache:
    """codes[b][h] etc. as float64 tensors; a copy of a GPU cache's state, or empty."""

    def __init__(self, B, H, d, cap, group, kv):
        self.B, self.H, self.d, self.cap, self.G, self.kv = B, H, d, cap, group, kv
        z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
        self.K, self.V = z(B, H, cap, d), z(B, H, cap, d)
        self.K_scale, self.V_scale = z(B, H, cap // BLOCK), z(B, H, cap // BLOCK)
        self.pos, self.score = torch.full((B, H, cap), -1, dtype=torch.int64), z(B, H, cap)
        self.score_tol = z(B, H, cap)

    def _quantise(self, codes, scale, x, a, b):
        """Rows x [b - a, d] into entries a .. b-1 of one head."""
        for j in range(a // BLOCK, (b + BLOCK - 1) // BLOCK):
            lo, hi = max(a, j * BLOCK), min(b, (j + 1) * BLOCK)
            if lo >= hi:
                continue
            new = x[lo - a : hi - a]
            fine = new[torch.isfinite(new)].abs()
            before = float(scale[j]) if j * BLOCK < a else 0.0
            after = max(before, pow2_scale(float(fine.max()) if fine.numel() else 0.0, self.kv))
            if before and after > before:
                codes[j * BLOCK : lo] = round_code(codes[j * BLOCK : lo] * (before / after), self.kv)
            new = torch.where(new.isnan(), 0.0, (new / after).clamp(-LIMIT[self.kv], LIMIT[self.kv]))
            codes[lo:hi] = round_code(new, self.kv)
            scale[j] = after

    def append(self, k, v, lens, counts=None, position=None, score=None):
        """k, v [B, H, n, d] (any float type, on any device)."""
        k, v = k.detach().cpu().double(), v.detach().cpu().double()
        n = k.shape[2]
        for b in range(self.B):
            a, c = lens[b], n if counts is None else counts[b]
            if a < 0 or c < 0 or c > n or a + c > self.cap:
                continue
            for h in range(self.H):
                self._quantise(self.K[b, h], self.K_scale[b, h], k[b, h, :c], a, a + c)
                self._quantise(self.V[b, h], self.V_scale[b, h], v[b, h, :c], a, a + c)
                p = a if position is None else position[b]
                self.pos[b, h, a : a + c] = torch.arange(p, p + c)
                self.score[b, h, a : a + c] = 0.0 if score is None else score[b, h, :c].detach().cpu().double()
                self.score_tol[b, h, a : a + c] = 0.0

    def values(self, which, b, h, total):
        codes, scale = getattr(self, which)[b, h, :total], getattr(self, which + "_scale")[b, h]
        return codes * scale.repeat_interleave(BLOCK)[:total, None]

    def attend(self, q, lens, counts=None, causal=True, accumulate=True):
        """out, lse [B, H * G, n, (d)] with NaN in rows behind the counts, and the tolerances of both.

        Errors of the kernels, relative to exact arithmetic:
        logits: products of a bf16 query and a code are exact; their fp32 sum of d terms in any order, also one
          that truncates, is off by at most d 2^-23 sum|q_i k_i|; the scale factors add 4 half steps:
          e_s = 2^-23 (d sum|q_i k_i| + 4 |s|), taken with the row's largest |s| and sum
        weights: 2 e_s + 2^-21 (|s - top| + 8) for the difference to the maximum, the exponentials (2 units of
          2^-22 each) and their sum in fp32 partial sums
        out: the weights' error and one rounding of them to 16 bits (2^-11, absolute 2^-25 below f16's normal
          numbers) against sum w |v|, then one bf16 half step 2^-8
        """
        q = q.detach().cpu().double()
        B, H, G, n, d = self.B, self.H, self.G, q.shape[2], self.d
        out = torch.full((B, H * G, n, d), math.nan, dtype=torch.float64)
        lse = torch.full((B, H * G, n), math.nan, dtype=torch.float64)
        out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
        for b in range(B):
            c, total = n if counts is None else counts[b], lens[b]
            for h in range(H):
                K, V = self.values("K", b, h, total), self.values("V", b, h, total)
                for r in range(c * G):
                    t, hq = r // G, h * G + r % G
                    end = max(0, total - c + t + 1) if causal else total
                    if end == 0:
                        out[b, hq, t], lse[b, hq, t] = 0.0, -math.inf
                        continue
                    s = K[:end] @ q[b, hq, t] / math.sqrt(d)
                    size = float((K[:end].abs() @ q[b, hq, t].abs()).max()) / math.sqrt(d)
                    e_s = 2.0 ** -23 * (d * size + 4 * float(s.abs().max()))
                    L = torch.logsumexp(s, 0)
                    w = torch.exp(s - L)
                    # weights too small to matter may be off by their whole fp32 underflow
                    e_w = 2 * e_s + 2.0 ** -21 * (float((s - s.max()).abs().clamp(max=90).max()) + 8)
                    out[b, hq, t], lse[b, hq, t] = w @ V[:end], L
                    mass = w @ V[:end].abs()
                    out_tol[b, hq, t] = 2.0 ** -8 * out[b, hq, t].abs() + (e_w + 2.0 ** -11) * mass * (1 + 2.0 ** -7) + \
                        2.0 ** -24 * float(V[:end].abs().sum(0).max() if end else 0) * float(w.max()) + 1e-37
                    lse_tol[b, hq, t] = e_s + 2.0 ** -21 * (1 + abs(float(L)))
                    if accumulate:
                        self.score[b, h, :end] += w
                        self.score_tol[b, h, :end] += w * e_w + 2.0 ** -100
                if accumulate and total:
                    self.score_tol[b, h, :total] += 2.0 ** -23 * self.score[b, h, :total].abs()
        return out, lse, out_tol, lse_tol

    def step(self, q, k, v, lens, counts=None, position=None, accumulate=True):
        n = k.shape[2]
        self.append(k, v, lens, counts, position)
        total = [a + (n if counts is None else counts[b]) for b, a in enumerate(lens)]
        return self.attend(q, total, counts, True, accumulate)

    def evict(self, lens, k_heavy, k_local, n_sink=0, score_mode=0, position=None):
        k = k_heavy + k_local
        for b in range(self.B):
            n = lens[b]
            if n <= k or n > self.cap:
                continue
            p = n if position is None else position[b]
            for h in range(self.H):
                first = n - k_local
                key = self.score[b, h, :first].float()
                if score_mode:
                    key = key / (p - self.pos[b, h, :first]).clamp(min=1).float()
                key = [(1, 0.0) if int(self.pos[b, h, j]) < n_sink else (0, -math.inf if math.isnan(x) else x)
                       for j, x in enumerate(key.tolist())]
                best = sorted(range(first), key=lambda j: (key[j], j), reverse=True)[:k_heavy]
                mine = torch.tensor(sorted(best) + list(range(first, n)), dtype=torch.long)
                for which in ("K", "V"):
                    rows = self.values(which, b, h, n)[mine]
                    self._quantise(getattr(self, which)[b, h], getattr(self, which + "_scale")[b, h], rows, 0, k)
                for t in (self.pos, self.score, self.score_tol):
                    t[b, h, :k] = t[b, h, mine].clone()
        return [min(n, k) if 0 <= n <= self.cap else n for n in lens]


def load(ref: RefCache, cache):
    """Copy a GPU cache's state into the reference."""
    for n in ("K", "V", "K_scale", "V_scale", "score"):
        getattr(ref, n).copy_(getattr(cache, n).cpu().double())
    ref.pos.copy_(cache.pos.cpu().long())
    ref.score_tol.zero_()


def same_state(cache, ref: RefCache):
    """Codes, scales and positions equal, scores within what their sums may be off."""
    for n in ("K_scale", "V_scale"):
        assert torch.allclose(getattr(cache, n).cpu().double(), getattr(ref, n), rtol=0, atol=0, equal_nan=True), n
    for n in ("K", "V"):
        got = getattr(cache, n).cpu().double()
        bad = (got != getattr(ref, n)) & ~(got.isnan() & getattr(ref, n).isnan())
        assert not bad.any(), (n, bad.nonzero()[:4])
    assert torch.equal(cache.pos.cpu().long(), ref.pos)
    got = cache.score.cpu().double()
    bad = (got - ref.score).abs() > ref.score_tol
    bad &= ~(got.isnan() & ref.score.isnan())
    bad &= got != ref.score  # infinities
    assert not bad.any(), ("score", bad.nonzero()[:4], got[bad][:4], ref.score[bad][:4])


def close(got, want, tol, name):
    """Within tol where want is a number; NaN in want marks places that are not compared."""
    got = got.detach().cpu().double()
    live = ~want.isnan()
    same = got == want
    bad = live & ~same & ~((got - want).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
