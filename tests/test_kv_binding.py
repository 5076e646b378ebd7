"""What the binding of the cache calls refuses before the library sees it, on tensors that are nowhere (no GPU needed)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from speculative_decoding_verification_draft_gb300 import ssdv


@pytest.fixture
def lib(monkeypatch):
    """A library that must not be reached."""
    monkeypatch.setattr(ssdv, "lib", lambda: pytest.fail("the call went on to the library"))


def arguments(at="cuda:0", dtype=torch.bfloat16, **other):
    """cache, page table, lengths, rows: on `at`, but for those named in `other`."""
    shapes = dict(cache=((4, 2, 4, 18 * 64), torch.uint8), table=((3, 4), torch.int32), lens=((3,), torch.int32),
                  count=((3,), torch.int32), x=((3, 5, 2, 64), dtype), y=((3, 5, 2, 64), dtype),
                  lse=((3, 5, 2), torch.float32), ws=((1 << 20,), torch.uint8))
    with FakeTensorMode():
        return {name: torch.empty(shape, dtype=t, device=other.get(name, at)) for name, (shape, t) in shapes.items()}


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 100, -(1 << 31) - 1])
def test_windows_of_more_than_32_bits(lib, window):
    t = arguments()
    with pytest.raises(ValueError, match="window"):
        ssdv.kv_attention(t["cache"], t["table"], t["lens"], t["x"], window=window)
