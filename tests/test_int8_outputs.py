"""Which given outputs of the 8-bit head lie apart from what else a call touches: the
binding's check by itself, on host memory (CPU only)."""

import pytest
import torch

from rollout_logprob_consistency_amd.int8 import _apart

I8 = torch.int8


def refuses(out, other, width=None):
    try:
        _apart("out", out, dict(other=other), width)
    except ValueError as e:
        assert str(e) == "out must lie apart from other"
        return True
    return False


def test_rows_beside_each_other():
    buf = torch.zeros(4096, dtype=torch.uint8)
    f32 = lambda lo, n: buf[lo:lo + 4 * n].view(torch.float32)  # noqa: E731
    assert not refuses(f32(0, 8), f32(32, 8)) and not refuses(f32(32, 8), f32(0, 8))
    assert refuses(f32(0, 9), f32(32, 8)) and refuses(f32(32, 8), f32(0, 9))
    assert refuses(f32(0, 100), f32(40, 1)) and refuses(f32(40, 1), f32(0, 100))
    rows = buf[:1024].view(I8).view(8, 128)[:, :100]
    # From the first row's start to the last one's end.
    assert refuses(rows, f32(128 * 7 + 96, 1)) and not refuses(rows, f32(128 * 7 + 100, 1))
    assert refuses(rows, f32(104, 1))


def test_codes_reach_to_the_next_multiple_of_16():
    buf = torch.zeros(256, dtype=torch.uint8)
    codes = buf[:128].view(I8).view(4, 32)[:, :21]
    behind = buf[96 + 24:96 + 28].view(torch.float32)
    assert not refuses(codes, behind) and refuses(codes, behind, 32)
    assert not refuses(codes, buf[128:132].view(torch.float32), 32)
    one = buf[:5].view(I8).view(1, 5)
    assert refuses(one, buf[8:12].view(torch.float32), 16)
    assert not refuses(one, buf[16:20].view(torch.float32), 16)


@pytest.mark.parametrize("shape", [(0,), (0, 16), (4, 0)])
def test_nothing_reaches_nowhere(shape):
    buf = torch.zeros(64, dtype=torch.float32)
    empty = buf[:0].view(shape) if 0 in shape else buf
    assert not refuses(empty, buf) and not refuses(buf, empty)
