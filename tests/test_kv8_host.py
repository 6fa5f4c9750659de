"""Host-side checks of the rotation and the paged 8-bit cache's calls (no GPU): every
refusal comes back before any launch, and the Python helpers refuse tensors that do
not fit."""
import ctypes

import pytest
import torch

import __graft_entry__
import sequence_long_context_gb300 as usp
from sequence_long_context_gb300 import _lib

FAKE = 1 << 20  # a 256-byte aligned non-null address; never dereferenced
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def cache(**over):
    a = dict(k_codes=FAKE, k_exps=FAKE, v_codes=FAKE, v_exps=FAKE, page_table=FAKE, seq_lens=FAKE,
             B=2, max_pages=4, num_pages=8, page_size=64, Hkv=2, D=128)
    a.update(over)
    return _lib.Kv8CacheStruct(**a)


def addr(c):
    return ctypes.addressof(c) if c is not None else None


def append(lib, c, **over):
    a = dict(k=FAKE, v=FAKE, q=None, q_out=None, Hq=8, table=None, rows=256, R=128, inter=0,
             pos=None, cu=None, T=4, dtype=0, out=None)
    a.update(over)
    return lib.usp_kv8_append(addr(c), a["k"], a["v"], a["q"], a["q_out"], a["Hq"], a["table"],
                              a["rows"], a["R"], a["inter"], a["pos"], a["cu"], a["T"], a["dtype"],
                              a["out"], None)


def read(lib, c, **over):
    a = dict(start=None, T=4, k=FAKE, v=FAKE, dtype=0)
    a.update(over)
    return lib.usp_kv8_read(addr(c), a["start"], a["T"], a["k"], a["v"], a["dtype"], None)


def attn(lib, c, **over):
    a = dict(q=FAKE, out=FAKE, lse=FAKE, cu=None, T=1, max_new=0, Hq=8, scale=0.0, causal=1,
             window=0, sink=0, dtype=0, ws=FAKE, wsb=1 << 40)
    a.update(over)
    return lib.usp_attn_kv8(addr(c), a["q"], a["out"], a["lse"], a["cu"], a["T"], a["max_new"],
                            a["Hq"], a["scale"], a["causal"], a["window"], a["sink"], a["dtype"],
                            a["ws"], a["wsb"], None)


def rope(lib, **over):
    a = dict(x=FAKE, y=FAR, table=FAKE, rows=256, R=128, inter=0, inverse=0, B=1, S=256, H=4, D=128,
             cu=None, cp=4, layout=1, dtype=0)
    a.update(over)
    return lib.usp_rope(a["x"], a["y"], a["table"], a["rows"], a["R"], a["inter"], a["inverse"],
                        a["B"], a["S"], a["H"], a["D"], a["cu"], a["cp"], a["layout"], a["dtype"],
                        None)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(max_pages=-1), 1), (dict(num_pages=-1), 1),
    (dict(page_size=0), 1), (dict(page_size=48), 2), (dict(page_size=16), 2),
    (dict(page_size=256), 2), (dict(D=96), 2), (dict(B=70000), 2), (dict(Hkv=70000), 2),
    (dict(max_pages=(1 << 24) + 1), 2), (dict(num_pages=1 << 30, Hkv=2), 2),
    (dict(k_codes=None), 1), (dict(v_exps=None), 1), (dict(page_table=None), 1),
    (dict(seq_lens=None), 1), (dict(k_codes=FAKE + 8), 3), (dict(v_exps=FAKE + 4), 3),
    (dict(page_table=FAKE + 2), 3), (dict(seq_lens=FAKE + 1), 3)])
def test_every_call_checks_the_cache(lib, over, code):
    c = cache(**over)
    assert append(lib, c) == code
    assert read(lib, c) == code
    assert attn(lib, c) == code


def test_null_cache(lib):
    assert append(lib, None) == 1 and read(lib, None) == 1 and attn(lib, None) == 1


def test_no_sequences_is_a_no_op(lib):
    c = cache(B=0, seq_lens=None, page_table=None, num_pages=0, k_codes=None, k_exps=None,
              v_codes=None, v_exps=None)
    assert append(lib, c) == 0 and read(lib, c) == 0 and attn(lib, c) == 0
    assert append(lib, c, cu=FAKE) == 1 and attn(lib, c, cu=FAKE) == 1  # packed needs a sequence
    assert read(lib, cache(), T=0, k=None, v=None) == 0


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(T=(1 << 30) + 1), 2), (dict(dtype=7), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3), (dict(cu=FAKE + 2), 3),
    (dict(out=FAKE + 1), 3), (dict(q=FAR), 1), (dict(q_out=FAR), 1),
    (dict(q=FAR, q_out=FAR, Hq=0), 1), (dict(q=FAR, q_out=FAR, Hq=70000), 1),
    (dict(q=FAR + 8, q_out=FAR + 8), 3), (dict(q=FAR, q_out=FAR + 1024), 1),
    (dict(q=FAR, q_out=FAKE), 1), (dict(pos=FAKE + 2), 3),
    (dict(table=FAKE, R=24), 1), (dict(table=FAKE, R=144), 1), (dict(table=FAKE, R=0), 1),
    (dict(table=FAKE, rows=0), 1), (dict(table=FAKE + 4), 3),
    (dict(table=FAKE, rows=255), 1)])  # the cache has 256 rows
def test_append_refuses(lib, over, code):
    assert append(lib, cache(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(dtype=2), 1), (dict(k=None), 1), (dict(v=FAKE + 8), 3),
    (dict(start=FAKE + 2), 3)])
def test_read_refuses(lib, over, code):
    assert read(lib, cache(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=0), 1), (dict(Hq=0), 1), (dict(Hq=7), 1), (dict(sink=-1), 1), (dict(dtype=1), 2),
    (dict(dtype=9), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(lse=None), 1),
    (dict(q=FAKE + 8), 3), (dict(out=FAKE + 8), 3), (dict(lse=FAKE + 8), 3), (dict(cu=FAKE + 1), 3),
    (dict(ws=FAKE + 16), 3), (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(T=1 << 25), 2)])
def test_attn_refuses(lib, over, code):
    assert attn(lib, cache(max_pages=4096), **over) == code


def test_attn_workspace_sizes(lib):
    f = usp.usp_attn_kv8_workspace_size
    for mp, few in ((4, True), (4096, False)):  # 256 and 262144 rows of each sequence
        c = cache(max_pages=mp)
        for T, cu in ((1, None), (3, None), (300, None), (300, FAKE)):
            for max_new in (0, 2):
                need = f(2, T, max_new, cu is not None, mp * 64, 8, 2, 128)
                if few and (T < 300 or (cu and max_new)):
                    assert need == 0  # few rows, few keys
                    continue
                assert need > 0
                assert attn(lib, c, T=T, max_new=max_new, cu=cu, wsb=need - 1) == 4
                assert attn(lib, c, T=T, max_new=max_new, cu=cu, ws=None) == 4
    assert f(2, 0, 0, False, 256, 8, 2, 128) == 0 and f(2, 1, 0, False, 1 << 20, 7, 2, 128) == 0
    assert f(2, 1, 0, False, 1 << 20, 8, 2, 96) == 0 and f(2, 1 << 25, 0, False, 256, 8, 2, 128) == 0
    assert f(2, 1, 0, False, -1, 8, 2, 128) == 0 and f(2, 1, 0, False, (1 << 30) + 1, 8, 2, 128) == 0
    # dense calls do not look at max_new
    assert f(2, 300, 2, False, 256, 8, 2, 128) == f(2, 300, 0, False, 256, 8, 2, 128)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), 1), (dict(S=-4), 1), (dict(H=0), 1), (dict(cp=0), 1), (dict(table=None), 1),
    (dict(dtype=5), 1), (dict(layout=9), 1), (dict(D=96, R=64), 2), (dict(S=252), 1),
    (dict(layout=0, S=250), 1), (dict(R=8), 1), (dict(R=40), 1), (dict(R=144), 1), (dict(rows=255), 1),
    (dict(table=FAKE + 4), 3), (dict(x=None), 1), (dict(y=None), 1), (dict(x=FAKE + 2), 3),
    (dict(y=FAR + 8), 3), (dict(cu=FAKE + 2), 3), (dict(cu=FAKE, B=0), 1),
    (dict(y=FAKE + 256), 1)])  # partial overlap
def test_rope_refuses(lib, over, code):
    assert rope(lib, **over) == code


def test_rope_of_nothing(lib):
    assert rope(lib, S=0, x=None, y=None) == 0 and rope(lib, B=0, x=None, y=None) == 0


def test_rope_table():
    t = usp.rope_table(100000, 64, device="cpu")
    assert t.shape == (100000, 64) and t.dtype == torch.float32
    # angles of far positions in 64 bits: cos and sin to half a step of fp32
    p = torch.tensor([1, 777, 99999], dtype=torch.float64)
    a = p[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    want = torch.cat([a.cos(), a.sin()], -1)
    assert (t[p.long()].double() - want).abs().max() <= 2.0 ** -24
    assert torch.equal(usp.rope_table(9, 16, scale=0.5, device="cpu")[8], usp.rope_table(9, 16, device="cpu")[4])


def cpu_cache(**kw):
    return usp.kv8_cache(2, 100, 2, 64, device="cpu", **kw)


def test_cache_shapes():
    c = cpu_cache()
    assert c.k.shape == (4, 2, 64, 64) and c.k_exp.shape == (4, 2, 2) and c.page_table.tolist() == [[0, 1], [2, 3]]
    c = cpu_cache(page_size=128, num_pages=3)
    assert c.v.shape == (3, 2, 128, 64) and c.v_exp.shape == (3, 2, 4) and c.page_table.tolist() == [[-1], [-1]]
    assert c.seq_lens.tolist() == [0, 0]


@pytest.mark.parametrize("over", [
    dict(k=torch.zeros(4, 2, 64, 64)), dict(v=torch.zeros(3, 2, 64, 64, dtype=torch.uint8)),
    dict(k_exp=torch.zeros(4, 2, 1, dtype=torch.int8)), dict(k_exp=torch.zeros(4, 2, 2, dtype=torch.uint8)),
    dict(page_table=torch.zeros(2, dtype=torch.int32)), dict(page_table=torch.zeros(2, 2)),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)),
    dict(k=torch.zeros(4, 64, 2, 64, dtype=torch.uint8).transpose(1, 2))])
def test_helpers_refuse_a_cache_that_does_not_fit(over):
    c = cpu_cache()._replace(**over)
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros(2, 1, 2, 64, **bf)
    for call in (lambda: usp.kv8_append(c, k, k), lambda: usp.kv8_read(c, 1), lambda: usp.attn_kv8(k, c)):
        with pytest.raises(ValueError):
            call()


def test_helpers_refuse_arguments_that_do_not_fit():
    c = cpu_cache()
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    t = usp.rope_table(128, 64, device="cpu")
    for args, kw in [
            ((k.half(), k.half()), {}), ((k, k.float()), {}), ((k, k[:, :2]), {}),
            ((k[:1].contiguous(), k[:1].contiguous()), {}), ((k, k), dict(cu_seqlens=torch.zeros(3, **i32))),
            ((k[0], k[0]), {}), ((k[0], k[0]), dict(cu_seqlens=torch.zeros(2, **i32))),
            ((k, k), dict(q=k.float())), ((k, k), dict(q_out=k)), ((k, k), dict(q=k, q_out=k[:, :1])),
            ((k, k), dict(rope=t[:100])), ((k, k), dict(rope=t.double())), ((k, k), dict(rope=t[0])),
            ((k, k), dict(rope=t, positions=torch.zeros(2, 2, **i32))),
            ((k, k), dict(seq_lens_out=torch.zeros(2))),
            ((k.transpose(1, 2).contiguous().transpose(1, 2), k), {}),
            ((k, k), {})]:  # (a CPU tensor)
        with pytest.raises(ValueError):
            usp.kv8_append(c, *args, **kw)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    for x, kw in [(q.float(), {}), (q[0], {}), (q[:1], {}), (q[0], dict(cu_seqlens=torch.zeros(4, **i32)))]:
        with pytest.raises(ValueError):
            usp.attn_kv8(x, c, **kw)
    for x, kw in [(q.half(), {}), (q[0], {}), (q, dict(cu_seqlens=torch.zeros(2, **i32))),
                  (q, dict(out=q.float())), (q.transpose(1, 2), {}), (q, {})]:
        with pytest.raises(ValueError):
            usp.rope(x, t, **kw)
    with pytest.raises(ValueError):
        usp.rope(q, None)
    with pytest.raises(ValueError):
        usp.kv8_read(c, 3, dtype=torch.float16)
    with pytest.raises(ValueError):
        usp.kv8_read(c, 3, starts=torch.zeros(2))
