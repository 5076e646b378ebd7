"""What the binding of the cache calls refuses before the library sees it, on tensors that are nowhere (no GPU needed)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from speculative_decoding_verification_draft_gb300 import ssdv

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


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


@pytest.fixture
def first_device(monkeypatch):
    """cuda:0 is current, its current stream is 0 and in no capture."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)


def calls(t):
    return dict(
        append=lambda: ssdv.kv_append(t["cache"], t["table"], t["lens"], t["x"], t["y"], n_new=t["count"],
                                      workspace=t["ws"]),
        read=lambda: ssdv.kv_read(t["cache"], t["table"], t["lens"], 5, count=t["count"], out=(t["x"], t["y"]),
                                  workspace=t["ws"]),
        attention=lambda: ssdv.kv_attention(t["cache"], t["table"], t["lens"], t["x"], n_q=t["count"], out=t["y"],
                                            lse=t["lse"], workspace=t["ws"]))


@pytest.mark.parametrize("call,name", [(call, name) for call in ("append", "read", "attention")
                                       for name in ("table", "lens", "count", "x", "y", "ws")] + [("attention", "lse")])
def test_tensors_of_another_device(monkeypatch, first_device, call, name):
    class Library:
        def __getattr__(self, function):
            return lambda *a: pytest.fail(f"{function} was reached")
    monkeypatch.setattr(ssdv, "lib", Library)
    with pytest.raises(ValueError, match="the cache's device"):
        calls(arguments(**{name: "cuda:1"}))[call]()


@pytest.mark.parametrize("call", ["append", "read", "attention"])
def test_a_cache_that_is_not_on_the_current_device(lib, first_device, call):
    with pytest.raises(ValueError, match="current device"):
        calls(arguments(at="cuda:1"))[call]()


def test_a_stream_of_another_device(lib, first_device, monkeypatch):
    class Stream:
        cuda_stream, device = 7, torch.device("cuda:1")
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    t = arguments()
    with pytest.raises(ValueError, match="the stream on cuda:1"):
        ssdv.kv_append(t["cache"], t["table"], t["lens"], t["x"], t["y"], workspace=t["ws"], stream=Stream())


@pytest.mark.parametrize("call,what", [("append", "k and v"), ("read", "outputs"), ("attention", "q")])
def test_types_are_refused_by_name(monkeypatch, first_device, call, what):
    monkeypatch.setattr(ssdv, "lib", lambda: type("Library", (), {"__getattr__": lambda self, function: None})())
    with pytest.raises(TypeError, match=f"^{what} must be bfloat16 or float32, got torch.float16"):
        calls(arguments(dtype=torch.float16))[call]()
