"""An append and the attention behind it with nothing between them, where the attention
takes its units on one line (two dependent kernels): lengths that were 0 until the append
wrote them, and boundaries that were others until just before."""
import numpy as np
import pytest
import torch

import sequence_long_context_gb300 as usp
from tests._gpu import device

pytestmark = pytest.mark.gpu

BF, CAP, H, G, D = torch.bfloat16, 65536, 2, 4, 128


def tokens(dev, lead, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*lead, h, D, generator=g).to(BF).to(dev) for h in (H * G, H, H)]


def empty(dev, B, cap=CAP):
    return usp.kv8_cache(B, cap, H, D, page_size=64, num_pages=8 * B, device=dev)


def give_pages(c):
    """Eight pages (512 rows) to each sequence."""
    B = c.page_table.shape[0]
    c.page_table[:, :8] = torch.arange(8 * B, dtype=torch.int32, device=c.k.device).view(B, 8)
    return c


@pytest.mark.parametrize("B,T,cut", [
    (2, 1, None),    # lengths written in the append's launch
    (2, 16, None),
    (80, 80, list(range(81))),                               # .. by a kernel of their own
    (40, 100, np.minimum(100, 3 * np.arange(41)).tolist()),  # the last sequences bring nothing
])
def test_an_append_to_an_empty_cache_and_its_attention(B, T, cut):
    dev = device()
    q, k, v = tokens(dev, (B, T) if cut is None else (T,), T)
    cu, kw, last = None, {}, T
    if cut is not None:
        cu = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        kw = dict(cu_seqlens=cu, max_new=max(b - a for a, b in zip(cut, cut[1:])))
        new = torch.tensor(cut, dtype=torch.int32, device=dev)
        last = [b - a for a, b in zip(cut, cut[1:])]
    assert usp.usp_attn_kv8_workspace_size(B, T, kw.get("max_new", 0), cut is not None, CAP, H * G,
                                           H, D) > 0  # the line's partials

    def step(c, wait):
        if cut is not None:
            cu.copy_(new)
        wait()
        usp.kv8_append(c, k, v, cu_seqlens=cu)
        wait()
        return usp.attn_kv8(q, c, **kw)

    c = give_pages(empty(dev, B))
    want = step(c, torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert torch.isfinite(want[1]).all()  # every token sees at least itself
    assert c.seq_lens.tolist() == ([T] * B if cut is None else last)
    got = []
    for _ in range(20):
        c.seq_lens.zero_()
        if cut is not None:
            cu.zero_()
        got.append(step(c, lambda: None))
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    usp.usp_device_status()


def test_the_line_in_a_captured_step():
    """Append, then two dependent kernels, captured and replayed as the cache grows."""
    dev = device()
    B = 2
    a, b = (give_pages(empty(dev, B)) for _ in "ab")
    q, k, v = tokens(dev, (B, 1), 1)
    step = lambda c: (usp.kv8_append(c, k, v), usp.attn_kv8(q, c))[1]  # noqa: E731
    s = torch.cuda.Stream(device=dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(give_pages(empty(dev, B)))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(a)
    for i in range(70):
        for x, y in zip((q, k, v), tokens(dev, (B, 1), i + 2)):
            x.copy_(y)
        graph.replay()
        got = out.clone(), lse.clone()
        want = step(b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    assert a.seq_lens.tolist() == b.seq_lens.tolist() == [70, 70]


def test_a_captured_chunk_grows_the_cache():
    """An append of more than 64 tokens, whose lengths a second, dependent kernel writes in
    place, and the chunk's attention, captured and replayed."""
    dev = device()
    B, T = 2, 100
    a, b = (give_pages(empty(dev, B)) for _ in "ab")
    q, k, v = tokens(dev, (B, T), 1)
    table = usp.rope_table(CAP, D, device=dev)

    def step(c):
        _, qr = usp.kv8_append(c, k, v, q=q, rope=table)
        return usp.attn_kv8(qr, c)

    s = torch.cuda.Stream(device=dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(give_pages(empty(dev, B)))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(a)
    for i in range(5):
        for x, y in zip((q, k, v), tokens(dev, (B, T), i + 2)):
            x.copy_(y)
        graph.replay()
        got = out.clone(), lse.clone()
        want = step(b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    assert a.seq_lens.tolist() == b.seq_lens.tolist() == [500, 500]
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("packed", [False, True])
def test_an_empty_chunk_at_given_positions(packed):
    """No tokens: lengths stay, with a table of fewer positions than the cache has rows."""
    dev = device()
    c = give_pages(empty(dev, 2))
    c.seq_lens.copy_(torch.tensor([5, 0]))
    lead = (0,) if packed else (2, 0)
    q, k, v = tokens(dev, lead, 1)
    lens, qr = usp.kv8_append(c, k, v, q=q, rope=usp.rope_table(8, D, device=dev),
                              positions=torch.empty(lead, dtype=torch.int32, device=dev),
                              cu_seqlens=torch.zeros(3, dtype=torch.int32, device=dev) if packed else None)
    assert lens.tolist() == [5, 0] and qr.shape == q.shape
