"""GPU tests of every form of the sparse attention's kernel: CTAs of 2, 4 and 8 warps by how many tokens and cached heads a
call has, up to 8 query rows a cached head and more, both head sizes and codes; and outputs whose rows are not dense."""
from __future__ import annotations

import pytest
import torch

from h2o_heavy_hitter_decode_gb300 import H2OBlockCache  # noqa: F401  (the library is there)
from test_gpu_sparse import compare, filled, ints, rows

pytestmark = pytest.mark.gpu

DEV = "cuda"


def lens_of(B, cap):
    return [(29 * b + 11) % (cap + 1) for b in range(B)]


FORMS = [  # B, H, G, n, d, kv, cap, (n_blocks, n_first, n_last); warps of a CTA on 152 SMs
    (40, 8, 9, 1, 128, "e4m3", 128, (2, 0, 1)),     # 2, more than 8 rows
    (40, 8, 16, 1, 128, "int8", 128, (3, 1, 1)),
    (40, 8, 12, 1, 64, "e4m3", 160, (3, 1, 1)),
    (40, 8, 10, 1, 64, "int8", 128, (2, 0, 1)),
    (60, 2, 9, 3, 128, "int8", 128, (2, 0, 1)),     # of several tokens
    (31, 2, 33, 5, 64, "e4m3", 96, (2, 0, 1)),
    (310, 1, 71, 1, 64, "int8", 96, (2, 0, 1)),     # of more rows than keep their codes
    (310, 1, 71, 1, 128, "e4m3", 96, (2, 1, 1)),
    (20, 8, 9, 1, 128, "e4m3", 160, (3, 1, 1)),     # 4, more than 8 rows
    (20, 8, 16, 1, 128, "int8", 128, (2, 0, 1)),
    (20, 8, 13, 1, 64, "e4m3", 160, (3, 1, 1)),
    (60, 8, 3, 1, 128, "e4m3", 160, (3, 1, 1)),     # 2, up to 8 rows
    (60, 8, 8, 1, 128, "int8", 128, (2, 0, 1)),
    (60, 8, 5, 1, 64, "e4m3", 128, (3, 0, 1)),
    (60, 8, 1, 1, 64, "int8", 128, (3, 0, 1)),
    (40, 8, 3, 1, 128, "e4m3", 160, (3, 1, 1)),     # 4, up to 8 rows
    (40, 8, 8, 1, 128, "int8", 128, (2, 0, 1)),
    (40, 8, 5, 1, 64, "int8", 128, (3, 0, 1)),
    (20, 8, 2, 1, 128, "int8", 640, (6, 1, 2)),     # in clusters of two
    (20, 8, 2, 1, 64, "e4m3", 640, (6, 1, 2)),
    (4, 2, 9, 1, 64, "e4m3", 2048, (20, 1, 2)),     # 8, more than 8 rows, clusters
    (4, 2, 9, 1, 128, "int8", 2048, (20, 1, 2)),
]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_forms(case):
    B, H, G, n, d, kv, cap, choice = case
    lens = lens_of(B, cap)
    c, r, g = filled(51, B, H, d, cap, lens, G, n, kv)
    q = rows(g, B, H * G, n, d, scale=1.5)
    lse, blocks = torch.zeros(B, H * G, n, device=DEV), torch.zeros(B, H, n, choice[0], dtype=torch.int32, device=DEV)
    out = c.attend_sparse(q, ints(lens), *choice, lse=lse, blocks=blocks)
    compare(c, r, out, lse, blocks, r.attend_sparse(q, lens, *choice), choice[0])
    assert c.error_bits() == 0


@pytest.mark.parametrize("case", [(40, 8, 9, 1, 128, "e4m3", 128, (2, 0, 1)), (60, 8, 3, 1, 64, "int8", 160, (3, 1, 1)),
                                  (20, 8, 2, 1, 128, "e4m3", 640, (6, 1, 2)), (3, 2, 4, 3, 64, "int8", 512, (5, 1, 2))],
                         ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_steps_of_forms(case):
    B, H, G, n, d, kv, cap, choice = case
    lens = [min(a, cap - n) for a in lens_of(B, cap)]
    c, r, g = filled(52, B, H, d, cap, lens, G, n, kv)
    q, k, v = rows(g, B, H * G, n, d, "tokens"), rows(g, B, H, n, d, "tokens", 4.0), rows(g, B, H, n, d, "slice")
    lse, blocks = torch.zeros(B, H * G, n, device=DEV), torch.zeros(B, H, n, choice[0], dtype=torch.int32, device=DEV)
    out = c.step_sparse(q, k, v, ints(lens), *choice, lse=lse, blocks=blocks)
    compare(c, r, out, lse, blocks, r.step_sparse(q, k, v, lens, *choice), choice[0])
    assert c.error_bits() == 0


@pytest.mark.parametrize("layout", ["tokens", "slice"])
@pytest.mark.parametrize("case", [(3, 2, 4, 3, 128, "e4m3", 512, (5, 1, 2)), (2, 3, 11, 2, 64, "int8", 512, (5, 1, 2)),
                                  (40, 8, 9, 1, 128, "int8", 128, (2, 0, 1)), (60, 8, 3, 1, 64, "e4m3", 160, (3, 1, 1)),
                                  (20, 8, 2, 1, 128, "int8", 640, (6, 1, 2)), (1, 2, 8, 1, 64, "e4m3", 8192, (17, 1, 2))],
                         ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_outputs_whose_rows_are_not_dense(case, layout):
    """A view of token-first rows, and heads of wider rows: what lies between them stays as it was, as do rows behind a
    sequence's count."""
    B, H, G, n, d, kv, cap, choice = case
    lens, counts = lens_of(B, cap), [n - b % (n + 1) for b in range(B)]
    lens[0] = cap
    c, r, g = filled(53, B, H, d, cap, lens, G, n, kv)
    q = rows(g, B, H * G, n, d)
    wide = torch.full((B, n, H * G + (3 if layout == "slice" else 0), d + (16 if layout == "slice" else 0)), 5.0,
                      dtype=torch.bfloat16, device=DEV)
    out = (wide[:, :, 2:-1, 8:-8] if layout == "slice" else wide).transpose(1, 2)
    lse, blocks = torch.zeros(B, H * G, n, device=DEV), torch.zeros(B, H, n, choice[0], dtype=torch.int32, device=DEV)
    got = c.attend_sparse(q, ints(lens), *choice, counts=ints(counts), out=out, lse=lse, blocks=blocks)
    assert got is out
    want = r.attend_sparse(q, lens, *choice, counts)
    for b in range(B):
        assert bool((out[b, :, counts[b]:] == 5).all())
    compare(c, r, out, lse, blocks, want, choice[0])
    out.fill_(5.0)
    assert bool((wide == 5).all())
    assert c.error_bits() == 0
