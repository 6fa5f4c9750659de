"""Host-side checks of the 4-bit cache calls (no GPU): every refusal comes back
before any launch, and the Python helpers refuse tensors that do not fit."""
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


def cache(base=FAKE, **over):
    a = dict(k_codes=base, k_scales=base + (1 << 30), v_codes=base + (2 << 30),
             v_scales=base + (3 << 30), key_weight=base + (4 << 30), seq_lens=base + (5 << 30), B=2,
             capacity=64, Hkv=2, D=128, k_descale=1.0, v_descale=1.0)
    a.update(over)
    return _lib.Kv4CacheStruct(**a)


BAD_CACHE = [
    (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(capacity=-16), 1), (dict(capacity=72), 1),
    (dict(D=96), 2), (dict(B=70000), 2), (dict(Hkv=70000), 2),
    (dict(k_descale=0.0), 1), (dict(v_descale=-1.0), 1), (dict(k_descale=float("nan")), 1),
    (dict(v_descale=float("inf")), 1), (dict(k_descale=1e-39), 1),
    (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(seq_lens=None), 1),
    (dict(k_codes=FAKE + 8), 3), (dict(v_scales=FAKE + 4), 3), (dict(key_weight=FAKE + 4), 3),
    (dict(seq_lens=FAKE + 2), 3),
]


def append(lib, c, **over):
    a = dict(k=FAKE, v=FAKE, w=None, cu=None, T=4, dtype=0, out=None)
    a.update(over)
    return lib.usp_kv4_append(ctypes.addressof(c) if c is not None else None, a["k"], a["v"],
                              a["w"], a["cu"], a["T"], a["dtype"], a["out"], None)


def read(lib, c, **over):
    a = dict(start=None, T=4, k=FAKE, v=FAKE, dtype=0)
    a.update(over)
    return lib.usp_kv4_read(ctypes.addressof(c) if c is not None else None, a["start"], a["T"],
                            a["k"], a["v"], a["dtype"], None)


def decode(lib, c, **over):
    a = dict(q=FAKE, out=FAKE, lse=FAKE, Tq=1, Hq=8, scale=0.0, causal=1, window=0, sink=0, acc=0,
             dtype=0, ws=FAKE, wsb=1 << 40)
    a.update(over)
    return lib.usp_attn_decode_kv4(
        ctypes.addressof(c) if c is not None else None, a["q"], a["out"], a["lse"], a["Tq"],
        a["Hq"], a["scale"], a["causal"], a["window"], a["sink"], a["acc"], a["dtype"], a["ws"],
        a["wsb"], None)


def evict(lib, c, d, **over):
    a = dict(kept=FAR, keep=32, recent=4, sink=2)
    a.update(over)
    return lib.usp_kv4_evict(ctypes.addressof(c), ctypes.addressof(d), a["kept"], a["keep"],
                             a["recent"], a["sink"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE)
def test_every_call_checks_the_cache(lib, over, code):
    c = cache(**over)
    assert append(lib, c) == code
    assert read(lib, c) == code
    assert decode(lib, c) == code
    assert evict(lib, c, c) == code
    assert evict(lib, cache(base=FAR), c) == code


def test_null_cache(lib):
    assert append(lib, None) == 1 and read(lib, None) == 1 and decode(lib, None) == 1


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(dtype=7), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3), (dict(w=FAKE + 2), 3), (dict(cu=FAKE + 2), 3),
    (dict(out=FAKE + 1), 3)])
def test_append_refuses(lib, over, code):
    assert append(lib, cache(), **over) == code


def test_append_refuses_weights_without_a_place(lib):
    assert append(lib, cache(key_weight=None), w=FAKE) == 1
    assert append(lib, cache(B=0, seq_lens=None), cu=FAKE) == 1  # packed needs a sequence


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(dtype=2), 1), (dict(k=None), 1), (dict(v=FAKE + 8), 3),
    (dict(start=FAKE + 2), 3)])
def test_read_refuses(lib, over, code):
    assert read(lib, cache(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(Tq=0), 1), (dict(Hq=0), 1), (dict(Hq=7), 1), (dict(sink=-1), 1), (dict(dtype=1), 2),
    (dict(dtype=9), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(lse=None), 1),
    (dict(q=FAKE + 8), 3), (dict(out=FAKE + 8), 3), (dict(lse=FAKE + 8), 3),
    (dict(ws=FAKE + 16), 3), (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(Tq=1 << 20), 2)])
def test_decode_refuses(lib, over, code):
    assert decode(lib, cache(), **over) == code


def test_decode_accumulate_needs_weights(lib):
    assert decode(lib, cache(key_weight=None), acc=1) == 1


def test_decode_workspace_sizes(lib):
    f = usp.usp_attn_decode_kv4_workspace_size
    plain, acc = f(2, 1, 64, 8, 2, 128, 0), f(2, 1, 64, 8, 2, 128, 1)
    assert plain >= (304 + 4) * 8 * 128 * 4
    assert acc >= plain + 2 * 2 * 64 * 4 * 4
    assert f(2, 0, 64, 8, 2, 128, 0) == 0 and f(2, 1, 64, 7, 2, 128, 0) == 0
    assert decode(lib, cache(), wsb=plain - 1) == 4
    assert decode(lib, cache(), acc=1, wsb=acc - 1) == 4


@pytest.mark.parametrize("over,code", [
    (dict(keep=0), 1), (dict(recent=-1), 1), (dict(sink=-1), 1), (dict(recent=31), 1),
    (dict(keep=65), 1), (dict(kept=None), 1), (dict(kept=FAR + 4), 3),
    (dict(recent=2**31 - 1, sink=2**31 - 1), 1)])
def test_evict_refuses(lib, over, code):
    assert evict(lib, cache(), cache(), **over) == code


def test_evict_refuses_caches_that_do_not_fit_or_overlap(lib):
    src = cache()
    for over in (dict(B=1), dict(Hkv=1), dict(D=64)):
        assert evict(lib, src, cache(base=FAR, **over), kept=1 << 45) == 1
    assert evict(lib, cache(key_weight=None), cache(base=FAR), kept=1 << 45) == 1
    # shares one array, or part of one, with the source
    assert evict(lib, src, cache(base=FAR, v_codes=FAKE + (2 << 30)), kept=1 << 45) == 1
    assert evict(lib, src, cache(base=FAR, k_codes=FAKE + 4096), kept=1 << 45) == 1
    assert evict(lib, src, cache(base=FAR, seq_lens=src.seq_lens), kept=1 << 45) == 1
    assert evict(lib, src, cache(base=FAR), kept=FAKE) == 1
    # in place means every pointer
    assert evict(lib, src, cache(key_weight=None), kept=FAR) == 1


def test_evict_in_place_refuses_a_list_inside_the_cache(lib):
    c = cache()
    for at in (c.k_codes, c.v_scales + 512, c.key_weight + 512, c.seq_lens):  # (arrays of 1 KB)
        assert evict(lib, c, c, kept=at) == 1


def test_nothing_to_do(lib):
    none = dict(k_codes=None, k_scales=None, v_codes=None, v_scales=None, key_weight=None,
                seq_lens=None, B=0)
    n0 = lib.usp_launch_count()
    c = cache(**none)
    assert append(lib, c, k=None, v=None) == 0
    assert read(lib, c, k=None, v=None) == 0
    assert decode(lib, c, q=None, out=None, lse=None, ws=None, wsb=0) == 0
    assert evict(lib, c, c, kept=None) == 0
    assert read(lib, cache(), T=0, k=None, v=None) == 0
    assert lib.usp_launch_count() == n0


def weights(lib, **over):
    a = dict(q=FAKE, k=FAKE, lse=FAKE, w=FAKE, B=1, S=256, Hq=4, Hkv=2, D=64, causal=1, window=0,
             sink=0, cu=None, cp=4, layout=1, observe=0, dtype=0, flags=0, ws=None, wsb=0)
    a.update(over)
    return lib.usp_attn_key_weights(a["q"], a["k"], a["lse"], a["w"], a["B"], a["S"], a["Hq"],
                                    a["Hkv"], a["D"], 0.0, a["causal"], a["window"], a["sink"],
                                    a["cu"], a["cp"], a["layout"], a["observe"], a["dtype"],
                                    a["flags"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(Hq=3), 1), (dict(D=96), 2), (dict(S=255), 1), (dict(cp=0), 1), (dict(layout=5), 1),
    (dict(sink=-1), 1), (dict(dtype=4), 1), (dict(flags=4), 2), (dict(flags=2), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(lse=None), 1), (dict(w=None), 1),
    (dict(q=FAKE + 8), 3), (dict(w=FAKE + 4), 3), (dict(ws=FAKE + 8), 3),
    (dict(S=8192), 4)])
def test_key_weights_refuses(lib, over, code):
    assert weights(lib, **over) == code


def test_key_weights_workspace(lib):
    f = usp.usp_attn_key_weights_workspace_size
    n = f(1, 8192, 32, 8, 0, torch.bfloat16)
    assert n > 0 and n % (8192 * 8 * 4) == 0
    assert weights(lib, S=8192, Hq=32, Hkv=8, ws=FAKE, wsb=n - 1) == 4
    assert f(1, 8192, 32, 8, 0, torch.float32) == 0           # one pass, no parts
    assert f(1, 8192, 32, 8, 0, torch.bfloat16, usp.FLAG_FORCE_SIMT) == 0
    assert f(-1, 8192, 32, 8, 0, torch.bfloat16) == 0 and f(1, 8192, 7, 8, 0, torch.bfloat16) == 0
    assert weights(lib, S=0, q=None, k=None, lse=None, w=None) == 0


def test_key_weights_of_very_long_prompts_are_cut(lib):
    """An item's roles wait for one another for at most 2 s, and a pair of a query
    tile and a head takes 1.2 us: items have 2^18 pairs at most, so the parts are
    tiles x heads / 2^18 (each [B, Hkv, S] fp32)."""
    f = usp.usp_attn_key_weights_workspace_size
    assert f(1, 2 ** 20, 32, 1, 0, torch.bfloat16) == 0                    # 2^18 pairs
    assert f(1, 2 ** 21, 128, 1, 0, torch.bfloat16) == 8 * 2 ** 21 * 4     # 2^21
    assert f(1, 2 ** 22, 16, 1, 0, torch.bfloat16) == 2 * 2 ** 22 * 4      # 2^19
    assert f(1, 2 ** 22, 16, 1, 4096, torch.bfloat16) == 0                 # few queries


def test_helpers_refuse_what_does_not_fit():
    c = usp.kv4_cache(2, 40, 2, 128, device="cpu", key_weight=True)
    assert c.k.shape == (2, 2, 48, 64) and c.v_scale.shape == (2, 2, 48, 4)
    k = torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16)
    bad = [
        lambda: usp.kv4_append(c, k.half(), k.half()),
        lambda: usp.kv4_append(c, k, k.float()),
        lambda: usp.kv4_append(c, k[:1], k),
        lambda: usp.kv4_append(c, k.transpose(1, 2).contiguous().transpose(1, 2), k),
        lambda: usp.kv4_append(c, k, k, key_weight=torch.zeros(2, 2, 4)),
        lambda: usp.kv4_append(c._replace(key_weight=None), k, k, key_weight=torch.zeros(2, 2, 3)),
        lambda: usp.kv4_append(c, k, k, seq_lens_out=torch.zeros(2, dtype=torch.int64)),
        lambda: usp.kv4_append(c, k[0], k[0], cu_seqlens=torch.zeros(2, dtype=torch.int32)),
        lambda: usp.kv4_append(c._replace(v=c.v[:, :, :32]), k, k),
        lambda: usp.kv4_append(c._replace(k_scale=c.k_scale[..., :2]), k, k),
        lambda: usp.kv4_append(c._replace(seq_lens=c.seq_lens.long()), k, k),
        lambda: usp.kv4_read(c, 4, starts=torch.zeros(3, dtype=torch.int32)),
        lambda: usp.kv4_read(c, 4, dtype=torch.float16),
        lambda: usp.attn_decode_kv4(torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), c),
        lambda: usp.attn_decode_kv4(torch.zeros(2, 1, 4, 128), c),
        lambda: usp.attn_decode_kv4(k, c._replace(key_weight=None), accumulate=True),
        lambda: usp.kv4_evict(c._replace(key_weight=None), 4),
        lambda: usp.kv4_evict(c, 0),
        lambda: usp.kv4_evict(c, 4, out=c._replace(k_descale=2.0)),
        lambda: usp.attn_key_weights(k, k, torch.zeros(2, 2, 4)),
        lambda: usp.attn_key_weights(k, k.float(), torch.zeros(2, 2, 3)),
        lambda: usp.attn_key_weights(k, k, torch.zeros(2, 2, 3, dtype=torch.float64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, KeyError)):
            f()
            pytest.fail(f"case {i} was accepted")


def test_capacities_whose_counts_would_pass_31_bits_are_refused(lib):
    """Such a cache (one sequence, one head of 64: 146 GB) fits the GPU."""
    for capacity in (2 ** 31 - 16, 2 ** 31 - 2 ** 20 + 16):
        c = cache(B=1, Hkv=1, D=64, capacity=capacity)
        assert append(lib, c) == read(lib, c) == 2
        assert decode(lib, c, Hq=1) == decode(lib, c, Hq=1, acc=1) == evict(lib, c, c) == 2


def test_workspace_size_is_0_for_what_the_decode_refuses(lib):
    f = usp.usp_attn_decode_kv4_workspace_size
    ok = dict(B=2, Tq=1, capacity=64, Hq=8, Hkv=2, D=128, accumulate=1)
    assert f(**ok) > 0 and f(**{**ok, "B": 0}) >= 0
    for bad in (dict(D=96), dict(capacity=72), dict(capacity=2 ** 31 - 16), dict(B=70000),
                dict(Hkv=70000, Hq=70000), dict(Tq=1 << 20), dict(B=65535, Hkv=65535, Hq=65535)):
        assert f(**{**ok, **bad}) == 0, bad


@pytest.mark.parametrize("over", [dict(v_descale="1"), dict(k_descale=None)])
def test_helpers_refuse_descales_that_are_no_numbers(over):
    c = usp.kv4_cache(2, 48, 2, 128, device="cpu", key_weight=True)._replace(**over)
    x = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16)
    for f in (lambda: usp.kv4_append(c, x, x), lambda: usp.kv4_read(c, 1),
              lambda: usp.attn_decode_kv4(x, c), lambda: usp.kv4_evict(c, 4)):
        with pytest.raises(ValueError, match="descale"):
            f()


@pytest.mark.parametrize("shape", [(3,), (2, 3), (2, 3, 2)])
def test_append_refuses_other_ranks(shape):
    c = usp.kv4_cache(2, 48, 2, 128, device="cpu")
    x = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        usp.kv4_append(c, x, x)


def test_permute_of_one_number_per_token_refuses(lib):
    def f(kind, B, S, H, D, eb, dst=FAR):
        return lib.usp_permute(FAKE, dst, kind, 1, B, S, H, D, 4, 1, eb, None)
    assert f(1, 2, 128, 1, 2, 4) == 1             # 8 bytes
    assert f(1, 2, 124, 1, 1, 4) == 1             # S % (2 cp)
    assert f(2, 2, 128, 1, 1, 4) == 1             # the Ulysses exchange moves whole heads
    assert f(1, 2, 128, 1, 1, 4, FAR + 4) == 3
    assert f(0, 65536, 1 << 15, 1, 1, 4) == 2     # 2^31 rows
    assert f(1, 0, 128, 1, 1, 4) == 0             # nothing to do
