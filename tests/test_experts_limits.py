"""Sizes at the ends of the experts' operators' ranges, without a GPU."""
import pytest
import torch

from nvfp4_w4a4_expert_amd import _lib as L
from nvfp4_w4a4_expert_amd import experts as X

BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def meta(*shape, dtype=BF16):
    """A tensor of any size without memory."""
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 6])
def test_row_counts_past_32_bits_are_refused(rows):
    o = meta(2, dtype=I32)
    f8 = lambda *s: (meta(*s, dtype=U8), meta(*s[:-1], 1, dtype=U8))
    for call in (lambda: X.grouped_linear(meta(4, 32), meta(1, rows, 32), o), lambda: X.grouped_linear(f8(4, 32), f8(1, rows, 32), o),
                 lambda: X.grouped_linear(meta(rows, 32), meta(1, 8, 32), o),
                 lambda: X.grouped_linear(meta(4, 32), meta(1, 8, 32), o, index=meta(rows, dtype=I32)),
                 lambda: X.route(meta(rows, 8, dtype=torch.float32), 2), lambda: X.permute(meta(rows // 2, 2, dtype=I32), 8),
                 lambda: X.combine(meta(rows, 32), meta(4, 2, dtype=torch.float32), meta(8, dtype=I32))):
        with pytest.raises(L.NVFP4Error) as e:
            call()
        assert e.value.status == L.ERR_UNSUPPORTED


def test_last_row_count_of_32_bits_reaches_the_device_check():
    with pytest.raises(ValueError, match="on a GPU"):
        X.grouped_linear(meta(4, 32), meta(1, 2 ** 31 - 1, 32), meta(2, dtype=I32))
