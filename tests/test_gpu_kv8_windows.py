"""Attention to the paged 8-bit cache with windows and sinks that reach far beyond any
sequence: what a caller passes for "no limit"."""
import pytest
import torch

import sequence_long_context_gb300 as usp
from tests import _kv8
from tests._gpu import device
from tests.test_gpu_kv8 import random_cache

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1


# lengths that are no multiple of 128; few rows (in clusters, and on one line) and chunks
@pytest.mark.parametrize("T,cap,lens", [(1, 2048, [1000, 77]), (3, 40960, [1000, 777]),
                                        (100, 2048, [1000, 333]), (300, 1024, [1000, 170])])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,sink", [(FAR, 0), (FAR, 5), (2 ** 31 - 900, 0), (2 ** 30 + 7, FAR),
                                         (50, FAR)])
def test_a_window_beyond_every_length_hides_nothing(T, cap, lens, causal, window, sink):
    dev = device()
    c = random_cache(dev, 2, cap, 2, 128, 64, lens, seed=T)
    q = torch.randn(2, T, 8, 128, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(dev)
    out, lse = usp.attn_kv8(q, c, causal=causal, window=window, sink_tokens=sink)
    _kv8.check(q, c, out, lse, causal, window, sink)
    want = usp.attn_kv8(q, c, causal=causal)  # the same keys in the same steps
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    usp.usp_device_status()
