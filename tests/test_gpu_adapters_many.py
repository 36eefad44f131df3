"""The launch that computes V for many rows, against float64 at depths where several CTAs share
K, the ring comes round and the adapters of a tile take several passes."""
import pytest

import adapters_ref as ref
import dense_gemm_persistent_gb300 as dg
from test_gpu_adapters import F32, Problem, close

pytestmark = pytest.mark.gpu


# 1100 rows are 9 tiles: 8 CTAs share 17 stages of K = 2056, 4 share 9 of 1032, 2 share 5 of 520, one has 3 of 264.
# A pass has 256 / r adapters (1 or 2 of rank 128, 16 of rank 16). The bounds are those of adapters_ref.py, of which the
# sum over K has the most: (K / 8 + 8) 2^-23 of the terms' magnitudes.
@pytest.mark.parametrize("K", [264, 520, 1032, 2056])
@pytest.mark.parametrize("r,L", [(16, 5), (16, 40), (72, 7), (128, 40)])
@pytest.mark.parametrize("order", ["mixed", "runs", "one"])
def test_v_of_many_rows(K, r, L, order):
    p = Problem(1100, 136, K, r, L, order=order, with_scale=order != "one")
    want = ref.adapters(p.X, p.A, p.B, p.ids, C=p.C, scale=p.scale, out_dtype=F32)
    for form in (0, 1):
        with dg.overrides(cta_pair=form):
            close(p.add("none", F32, F32), want)


@pytest.mark.parametrize("T,K,r,L", [(1025, 4096, 32, 9), (2500, 776, 64, 12), (20000, 136, 8, 30)])
def test_other_numbers_of_tiles(T, K, r, L):
    p = Problem(T, 40, K, r, L, order="runs")
    close(p.add("none", F32, F32), ref.adapters(p.X, p.A, p.B, p.ids, C=p.C, scale=p.scale, out_dtype=F32))
