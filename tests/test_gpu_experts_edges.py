"""The routed-FFN operators on the GPU at the edges of their types, sizes and
launches (bounds as in test_gpu_experts.py)."""
import numpy as np
import pytest
import torch

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
