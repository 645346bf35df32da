"""The routed-FFN operators on the GPU at the edges of their types, sizes and
launches (bounds as in test_gpu_experts.py)."""
import numpy as np
import pytest
import torch

from launches import launches
from oracle import experts_oracle as O

pytestmark = pytest.mark.gpu
P = pytest.importorskip("free_ffn_activation_amd.prox")

FP8 = torch.float8_e4m3fn


# --------------------------------------------------------------- quantizer
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_where_the_scale_is_a_few_subnormal_steps(block_rows):
    """amax / 448 of a few steps of 2^-149 is rounded down by up to a third: the
    quotients beyond 448 are held there (a NaN code would take a whole product row
    with it).  The values are exact in fp32, so codes and scales are those of the
    definition."""
    steps = [1, 100, 223, 224, 225, 448, 464, 465, 642, 671, 672, 673, 1000, 1120, 3568, 5709, 6049, 2 ** 13, 448 * 2 ** 12]
    g = np.random.default_rng(0)
    x = np.zeros((len(steps) * block_rows, 144), np.float32)
    for i, n in enumerate(steps):
        part = g.integers(-n, n + 1, (block_rows, 144))
        part[-1, 3], part[0, 130], part[-1, 143] = n, -n, n // 3
        x[i * block_rows:(i + 1) * block_rows] = part * 2.0 ** -149
    q = torch.empty(x.shape, device="cuda", dtype=FP8)
    scale = torch.empty(len(steps), 2, device="cuda")
    P.prox_fp8_quantize(torch.from_numpy(x).cuda(), q, scale, block_rows=block_rows)
    rq, rs = O.quantize(x, block_rows)
    assert np.array_equal(scale.cpu().numpy(), rs)
    got = q.float().cpu().numpy().astype(np.float64)
    assert not np.isnan(got).any()
    assert np.array_equal(got, rq)
    assert abs(rq).max() == 448


# ---------------------------------------------------------------- products
def codes(g, shape, subnormal):
    """Random e4m3 codes, none of them NaN; subnormal: that share of them 0 to 7."""
    c = g.integers(0, 256, shape)
    c = np.where(g.random(shape) < subnormal, c & 0x87, c)
    c = np.where((c & 0x7F) == 0x7F, 0, c).astype(np.uint8)
    return torch.from_numpy(c).cuda().view(FP8)


@pytest.mark.parametrize("subnormal", [0.0, 0.5, 0.9])
@pytest.mark.parametrize("rows,n,k", [(5, 40, 144), (130, 600, 128), (70, 130, 1040)])
def test_e4m3_products_are_cut_as_stated(rows, n, k, subnormal):
    """fp32 results of e4m3 products against the rule by which the matrix cores cut
    small products: what is left is added in fp32, (K + 8) 2 EPS of the magnitudes.
    Codes over the whole range: where the cut counts most, it is a thousand times
    that.  Scales of one."""
    g = np.random.default_rng(rows + n)
    a, w = codes(g, (rows, k), subnormal), codes(g, (1, n, k), subnormal)
    e = P.ProxExperts(w, scale=torch.ones(1, -(-n // 128), -(-k // 128), device="cuda"))
    out = torch.empty(rows, n, device="cuda")
    P.prox_grouped_matmul(e, a, out, a_scale=torch.ones(rows, -(-k // 128), device="cuda"))
    ha, hw = (t.float().cpu().numpy().astype(np.float64) for t in (a, w[0]))
    off = np.abs(out.cpu().numpy() - O.cut_product(ha, hw))
    assert (off <= (k + 8) * 2 * 2.0 ** -24 * (np.abs(ha) @ np.abs(hw).T)).all()


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("e", [5, 64, 65, 128])
def test_route_in_one_launch_is_one_block(e):
    """One block takes all tokens of such a call: a second one would do the same
    work again and write every output a second time, unordered."""
    i32 = dict(dtype=torch.int32, device="cuda")
    for t in (1, 16, 17, 32, 33, 47, 63, 64, 65):
        k = min(e, 8)
        bufs = (torch.zeros(t, e, device="cuda"), torch.empty(t, k, **i32), torch.empty(t, k, device="cuda"),
                torch.empty(e + 1, **i32), torch.empty(t * k, **i32), torch.empty(t, k, **i32),
                torch.empty(P.prox_expert_route_workspace_size(t, e, k), dtype=torch.uint8, device="cuda"))
        found = launches(lambda s: P.prox_expert_route(*bufs, stream=s))
        if t <= 64:
            assert len(found) == 1 and found[0][1] == 1, (t, found)
            assert "route_small_kernel" in found[0][0], found
        else:
            assert [f[1] for f in found] == [3, 3], (t, found)
