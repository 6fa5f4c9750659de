"""Attention and its gradients with windows and sinks that reach far beyond the sequence
(what a caller passes for "no limit"): they hide nothing."""
import pytest
import torch

import sequence_long_context_gb300 as usp
from tests._gpu import TOL, device

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1


@pytest.mark.parametrize("dtype,cp,ud,layout,cut", [
    (torch.bfloat16, 1, 1, "contiguous", None), (torch.bfloat16, 4, 1, "zigzag", None),
    (torch.bfloat16, 2, 2, "stripe", None), (torch.bfloat16, 1, 1, "contiguous", [0, 200, 640, 1024]),
    (torch.float32, 2, 1, "zigzag", None), (torch.float32, 1, 1, "contiguous", [0, 200, 640, 1024])])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,sink", [(FAR, 0), (FAR, FAR), (40, FAR), (2 ** 31 - 500, 7)])
def test_nothing_is_hidden(dtype, cp, ud, layout, cut, causal, window, sink):
    dev = device()
    g = torch.Generator().manual_seed(cp)
    lead = (2, 1024) if cut is None else (1024,)
    q, k, v, do = (torch.randn(*lead, h, 64, generator=g).to(dtype).to(dev) for h in (4, 2, 2, 4))
    cu = None if cut is None else torch.tensor(cut, dtype=torch.int32, device=dev)
    kw = dict(causal=causal, cu_seqlens=cu, cp=cp, ud=ud, layout=layout)
    out, lse = usp.attn_forward(q, k, v, window=window, sink_tokens=sink, **kw)
    want, wlse = usp.attn_forward(q, k, v, **kw)
    tol = TOL["bf16" if dtype is torch.bfloat16 else "fp32"]
    # (the order of the sums may differ with the mask's form)
    assert float((out.float() - want.float()).abs().max()) <= tol["o"]
    assert float((lse - wlse).abs().max()) <= tol["lse"]
    got = usp.attn_backward(q, k, v, out, lse, do, window=window, sink_tokens=sink, **kw)
    ref = usp.attn_backward(q, k, v, want, wlse, do, **kw)
    for a, b in zip(got, ref):
        assert float((a.float() - b.float()).norm()) <= tol["grad"] * float(b.float().norm())
    usp.usp_device_status()
