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
