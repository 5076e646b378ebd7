"""Windows that no context reaches: every one up to the largest int32 means "no window", on both attention kernels."""
import pytest
import torch

from test_gpu_kv_attention import check, ssdv  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("window", [1 << 30, 2 ** 31 - 33, 2 ** 31 - 32, 2 ** 31 - 5, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("past_only", [False, True])
@pytest.mark.parametrize("n,G,D,dtype", [(6, 2, 128, BF16), (6, 4, 128, BF16), (5, 8, 128, BF16), (32, 1, 128, BF16),
                                         (9, 8, 128, BF16), (6, 4, 64, F32)])
def test_windows_past_every_context(ssdv, n, G, D, dtype, window, past_only):  # noqa: F811
    check(ssdv, 2, 2, G, D, 32, dtype, n, [0, 130], window=window, past_only=past_only)
