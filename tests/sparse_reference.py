"""Sparse attention over blocks of a block-scaled cache in 64 bits on the CPU: bounds, the choice in whole numbers, and
attention over the chosen entries with the tolerances of block_reference.py."""
from __future__ import annotations

import math

import torch

from block_reference import BLOCK, RefCache, pow2_scale

UNIT = {"e4m3": 4.0, "int8": 1.0}


class SparseRef(RefCache):
    def bounds_of(self, b, h, total):
        """[blocks, 2, d] as int64: least and largest codes of the blocks of `total` entries."""
        out = []
        for j in range(0, total, BLOCK):
            rows = self.K[b, h, j : min(total, j + BLOCK)] / UNIT[self.kv]
            out.append(torch.stack([rows.amin(0).floor(), rows.amax(0).ceil()]))
        return torch.stack(out).long() if out else torch.zeros(0, 2, self.d, dtype=torch.int64)

    def choose(self, q, b, h, end, n_blocks, n_first, n_last, bounds):
        """Blocks of a token whose rows q [G, d] (float64) see `end` entries."""
        nb = -(-max(0, end) // BLOCK)
        if nb <= n_blocks:
            return list(range(nb))
        fine = q[torch.isfinite(q)].abs()
        scale = pow2_scale(float(fine.max()) if fine.numel() else 0.0, "int8")
        x = torch.round(torch.where(q.isnan(), 0.0, (q / scale).clamp(-127, 127))).long()
        m = (x[:, None] * torch.where(x[:, None] > 0, bounds[None, :nb, 1], bounds[None, :nb, 0])).sum(-1).amax(0)
        key = [float(m[j]) * float(self.K_scale[b, h, j]) for j in range(nb)]  # exact in 64 bits
        middle = sorted(range(n_first, nb - n_last), key=lambda j: (-key[j], j))
        wanted = n_blocks - n_first - n_last
        return sorted([*range(n_first), *middle[:wanted], *range(nb - n_last, nb)])

    def attend_sparse(self, q, lens, n_blocks, n_first, n_last, counts=None, causal=True, accumulate=True):
        """out, lse (NaN in rows behind the counts), their tolerances (derived as in RefCache.attend) and the lists of
        blocks: {(b, h, t): [..]}."""
        q = q.detach().cpu().double()
        B, H, G, n, d = self.B, self.H, self.G, q.shape[2], self.d
        out = torch.full((B, H * G, n, d), math.nan, dtype=torch.float64)
        lse = torch.full((B, H * G, n), math.nan, dtype=torch.float64)
        out_tol, lse_tol, lists = torch.zeros_like(out), torch.zeros_like(lse), {}
        for b in range(B):
            c, total = n if counts is None else counts[b], lens[b]
            if not (0 <= c <= n and 0 <= total <= self.cap):
                continue
            for h in range(H):
                bounds = self.bounds_of(b, h, total)
                K, V = self.values("K", b, h, total), self.values("V", b, h, total)
                touched = torch.zeros(self.cap, dtype=torch.float64)
                for t in range(c):
                    end = max(0, total - c + t + 1) if causal else total
                    rows = q[b, h * G : (h + 1) * G, t]
                    lists[b, h, t] = mine = self.choose(rows, b, h, end, n_blocks, n_first, n_last, bounds)
                    at = torch.tensor([j for i in mine for j in range(i * BLOCK, min(end, (i + 1) * BLOCK))], dtype=torch.long)
                    for g in range(G):
                        hq = h * G + g
                        if not len(at):
                            out[b, hq, t], lse[b, hq, t] = 0.0, -math.inf
                            continue
                        k, v = K[at], V[at]
                        if not torch.isfinite(rows[g]).all():
                            out[b, hq, t], lse[b, hq, t] = math.inf, math.inf  # stands for NaN: compared apart
                            if accumulate:
                                self.score[b, h, at] = math.nan
                            continue
                        s = k @ rows[g] / math.sqrt(d)
                        size = float((k.abs() @ rows[g].abs()).max()) / math.sqrt(d)
                        e_s = 2.0 ** -23 * (d * size + 4 * float(s.abs().max()))
                        L = torch.logsumexp(s, 0)
                        w = torch.exp(s - L)
                        e_w = 2 * e_s + 2.0 ** -21 * (float((s - s.max()).abs().clamp(max=90).max()) + 8)
                        out[b, hq, t], lse[b, hq, t] = w @ v, L
                        mass = w @ v.abs()
                        out_tol[b, hq, t] = 2.0 ** -8 * out[b, hq, t].abs() + (e_w + 2.0 ** -11) * mass * (1 + 2.0 ** -7) + \
                            2.0 ** -24 * float(v.abs().sum(0).max()) * float(w.max()) + 1e-37
                        lse_tol[b, hq, t] = e_s + 2.0 ** -21 * (1 + abs(float(L)))
                        if accumulate:
                            self.score[b, h, at] += w
                            self.score_tol[b, h, at] += w * e_w + 2.0 ** -100
                            touched[at] += 1
                self.score_tol[b, h] += torch.where(touched > 0, (1 + c) * 2.0 ** -23 * self.score[b, h].abs(), 0.0)
        return out, lse, out_tol, lse_tol, lists

    def step_sparse(self, q, k, v, lens, n_blocks, n_first, n_last, counts=None, position=None, accumulate=True):
        n = k.shape[2]
        self.append(k, v, lens, counts, position)
        total = [a + (n if counts is None else counts[b]) for b, a in enumerate(lens)]
        return self.attend_sparse(q, total, n_blocks, n_first, n_last, counts, True, accumulate)
