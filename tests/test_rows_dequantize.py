"""dequantize of 8-bit and 4-bit rows, without a GPU: every form against the formats'
definitions, experts' weights, results without rows."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_expert_amd import dense as D
from oracle import dense as OD

U8, F32 = torch.uint8, torch.float32


def codes_of(shape, seed):
    c = np.random.default_rng(seed).integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 0x7F) == 0x7F, 0, c).astype(np.uint8)


@pytest.mark.parametrize("shape", [(5, 64), (3, 5, 64), (64, 64, 64), (0, 64), (3, 0, 64)])
@pytest.mark.parametrize("scales", ["row", "mx"])
def test_fp8_rows(shape, scales):
    g = np.random.default_rng(1)
    c = codes_of(shape, 2)
    s = g.random(shape[:-1], np.float32) + 0.5 if scales == "row" else g.integers(120, 133, (*shape[:-1], shape[-1] // 32)).astype(np.uint8)
    got = D.FP8Rows(torch.from_numpy(c), torch.from_numpy(s)).dequantize()
    flat = OD.dequantize(c.reshape(-1, shape[-1]), s.reshape(-1) if scales == "row" else s.reshape(-1, shape[-1] // 32))
    assert got.dtype == F32 and got.shape == shape
    assert np.array_equal(got.numpy(), flat.astype(np.float32).reshape(shape))


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.mark.parametrize("rows", [0, 1, 7])
@pytest.mark.parametrize("scales", ["nv", "mx"])
@pytest.mark.parametrize("shape", [None, (), (1,), (1, 1, 1)])
def test_fp4_rows(rows, scales, shape):
    """Any number of rows; the scale of one element in any shape that linear takes."""
    K = 96
    c = np.random.default_rng(3).integers(0, 256, (rows, K // 2)).astype(np.uint8)
    if scales == "nv":
        s = codes_of((rows, K // 16), 4)
        each = np.repeat(OD.e4m3_decode(s), 16, axis=1)
    else:
        s = np.random.default_rng(5).integers(100, 150, (rows, K // 32)).astype(np.uint8)
        each = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)
    n = np.stack([c & 15, c >> 4], 2).reshape(rows, K)
    v = np.where(n & 8, -E2M1[n & 7], E2M1[n & 7]) * each * (1.0 if shape is None else 0.375)
    got = D.FP4Rows(torch.from_numpy(c), torch.from_numpy(s), None if shape is None else torch.full(shape, 0.375)).dequantize()
    assert got.dtype == F32 and got.shape == (rows, K) and np.array_equal(got.numpy(), v.astype(np.float32))
