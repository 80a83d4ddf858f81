"""GPU test of the block cache's operators in one run, as a layer of a decoding model uses them: prompts appended with
rotated keys, beams forked out of them, steps of rotated queries and keys over chosen blocks, beams reordered, an eviction,
dense steps behind it.  Rotated rows come from H2ORotary alone (tested against its formulas elsewhere); everything else is
compared with the 64-bit reference, as in the operators' own tests."""
from __future__ import annotations

import math

import pytest
import torch

from block_reference import BLOCK, close, load, same_state
from h2o_heavy_hitter_decode_gb300 import H2OBlockCache, H2ORotary
from sparse_reference import SparseRef

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(g, B, heads, n, d, scale=1.0):
    """A fused projection's token-first rows."""
    return (torch.randn(B, n, heads, d, generator=g, device=DEV) * scale).bfloat16().transpose(1, 2)


def copy_ref(to, source, parent, lens):
    """What H2OBlockCache.copy does: whole blocks."""
    for b, p in enumerate(parent):
        if p < 0:
            continue
        m = -(-lens[p] // BLOCK)
        for n in ("K", "V", "pos", "score", "score_tol"):
            getattr(to, n)[b, :, : m * BLOCK] = getattr(source, n)[p, :, : m * BLOCK]
        for n in ("K_scale", "V_scale"):
            getattr(to, n)[b, :, :m] = getattr(source, n)[p, :, :m]


@pytest.mark.parametrize("kv,d,axes,interleaved", [("e4m3", 128, 1, False), ("int8", 64, 3, True)])
@pytest.mark.parametrize("stream", ["current", "side"])
def test_layer(kv, d, axes, interleaved, stream):
    H, G, cap = 2, 3, 512
    g = torch.Generator(DEV).manual_seed(50)
    rotary = H2ORotary(d, axis=[i * axes // (d // 2) for i in range(d // 2)], interleaved=interleaved, eps=1e-6,
                       q_weight=torch.rand(d, generator=g, device=DEV) + 0.5, k_weight=torch.rand(d, generator=g, device=DEV) + 0.5)
    side = torch.cuda.Stream() if stream == "side" else torch.cuda.current_stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        # two prompts
        prompt, prompt_lens = H2OBlockCache(2, H, d, cap, kv=kv, bounds=True), [300, 171]
        k, v = rows(g, 2, H, 300, d), rows(g, 2, H, 300, d)
        first = torch.rand(2, H, 300, generator=g, device=DEV) * 5
        prompt.append(k, v, ints([0, 0]), counts=ints(prompt_lens), score=first, rotary=rotary)
        ref_prompt = SparseRef(2, H, d, cap, 1, kv)
        turned = rotary.apply(None, k, ints([0, 0]), ints(prompt_lens))[1]
        ref_prompt.append(turned, v, [0, 0], prompt_lens, None, first)
        ref_prompt.pos = torch.where(ref_prompt.pos < 0, prompt.pos.cpu().long(), ref_prompt.pos)
        same_state(prompt, ref_prompt)
        # three beams of the first, two of the second; a row that is free
        B = 6
        cache, ref = H2OBlockCache(B, H, d, cap, group=G, max_queries=2, kv=kv, bounds=True), SparseRef(B, H, d, cap, G, kv)
        load(ref, cache)
        parent = [0, 0, 0, 1, 1, -1]
        lengths = cache.copy(ints(parent), ints([0] * B), prompt, ints(prompt_lens))
        copy_ref(ref, ref_prompt, parent, prompt_lens)
        lens = [300, 300, 300, 171, 171, 0]
        assert lengths.tolist() == lens
        position = lengths.clone()
        for t in range(6):
            n = 1 + t % 2
            counts = [n] * 5 + [0]
            q, k, v = rows(g, B, H * G, n, d, 2.0), rows(g, B, H, n, d), rows(g, B, H, n, d)
            kept = q.clone(), k.clone()
            rq, rk = rotary.apply(q, k, position, ints(counts))
            lse = torch.zeros(B, H * G, n, device=DEV)
            if t < 4:
                blocks = torch.zeros(B, H, n, 6, dtype=torch.int32, device=DEV)
                out = cache.step_sparse(q, k, v, lengths, 6, 1, 2, counts=ints(counts), position=position, lse=lse,
                                        blocks=blocks, rotary=rotary)
                want, want_lse, tol, lse_tol, lists = ref.step_sparse(rq, rk, v, lens, 6, 1, 2, counts, position.tolist())
                for (b, h, i), mine in lists.items():
                    assert blocks[b, h, i].tolist() == mine + [-1] * (6 - len(mine))
            else:
                out = cache.step(q, k, v, lengths, counts=ints(counts), position=position, lse=lse, rotary=rotary)
                want, want_lse, tol, lse_tol = ref.step(rq, rk, v, lens, counts, position.tolist())
            assert torch.equal(q, kept[0]) and torch.equal(k, kept[1])
            close(out, want, tol, "out")
            close(lse, want_lse, lse_tol, "lse")
            same_state(cache, ref)
            lengths, position = lengths + ints(counts), position + ints(counts)
            lens = [a + c for a, c in zip(lens, counts)]
            if t in (0, 2):  # the better beams go on twice
                parent = [1, 1, 2, 4, 3, -1] if t == 0 else [2, 0, 0, -1, 3, -1]
                lengths = cache.copy(ints(parent), lengths)
                old = SparseRef(B, H, d, cap, G, kv)
                load_from(old, ref)
                copy_ref(ref, old, parent, lens)
                lens = [lens[p] if p >= 0 else lens[b] for b, p in enumerate(parent)]
                assert lengths.tolist() == lens
                position = position[ints([p if p >= 0 else b for b, p in enumerate(parent)]).long()].contiguous()
                same_state(cache, ref)
            if t == 3:
                load(ref, cache)  # the scores, to the bit, decide
                lengths = cache.evict(lengths, 60, 70, n_sink=4, position=position)
                lens = ref.evict(lens, 60, 70, 4, 0, position.tolist())
                assert lengths.tolist() == lens
                same_state(cache, ref)
            for b in range(B):
                for h in range(H):
                    want_bounds = ref.bounds_of(b, h, lens[b])
                    assert torch.equal(cache.bounds[b, h, : len(want_bounds)].cpu().long(), want_bounds)
        assert cache.error_bits() == 0 and prompt.error_bits() == 0


def load_from(to, source):
    for n in ("K", "V", "K_scale", "V_scale", "pos", "score", "score_tol"):
        getattr(to, n).copy_(getattr(source, n))


def test_rotation_in_a_captured_step():
    """One graph of rotation and sparse step, replayed at the positions of the moment."""
    g = torch.Generator(DEV).manual_seed(51)
    rotary = H2ORotary(64, dims=32, eps=1e-5)
    twins = [H2OBlockCache(2, 2, 64, 256, group=2, bounds=True) for _ in range(2)]
    lengths = ints([100, 37])
    k0, v0 = rows(g, 2, 2, 100, 64), rows(g, 2, 2, 100, 64)
    for c in twins:
        c.append(k0, v0, ints([0, 0]), counts=lengths, rotary=rotary)
    q, k, v = rows(g, 2, 4, 1, 64), rows(g, 2, 2, 1, 64), rows(g, 2, 2, 1, 64)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        twins[0].step_sparse(q, k, v, lengths, 3, out=out, rotary=rotary)
    torch.cuda.current_stream().wait_stream(side)
    want = twins[1].step_sparse(q, k, v, lengths, 3, rotary=rotary)
    assert torch.equal(out, want)
    with torch.cuda.graph(graph):
        twins[0].step_sparse(q, k, v, lengths, 3, out=out, rotary=rotary)
    for _ in range(3):
        lengths += 1
        q.copy_(rows(g, 2, 4, 1, 64)), k.copy_(rows(g, 2, 2, 1, 64))
        graph.replay()
        want = twins[1].step_sparse(q, k, v, lengths, 3, rotary=rotary)
        assert torch.equal(out, want)
        for n in ("K", "V", "score", "bounds", "pos"):
            assert torch.equal(getattr(twins[0], n).view(torch.uint8), getattr(twins[1], n).view(torch.uint8))
    assert math.isfinite(float(out.float().sum()))
