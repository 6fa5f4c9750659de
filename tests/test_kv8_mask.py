"""The mask arithmetic of the paged 8-bit cache's chunk kernel, compiled for the host, and
the mask's definition in Python's whole numbers: windows and sinks up to 2^31 - 1, cached
lengths up to 2^30, queries ahead of the first key."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sequence_long_context_gb300", "csrc")
SOURCE = """
#include "kv8_mask.h"
extern "C" uint32_t bits(int i, int len, int causal, int window, int sink, int k) {
  return usp::kv8::key_bits(usp::kv8::row_keys(i, len, causal, usp::kv8::window_of(window), sink), k);
}
"""


@pytest.fixture(scope="module")
def bits(tmp_path_factory):
    d = tmp_path_factory.mktemp("mask")
    (d / "mask.cpp").write_text(SOURCE)
    so = str(d / "mask.so")
    # (-fwrapv: what passes 32 bits wraps, as it does on the GPU)
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(d / "mask.cpp"),
                    "-o", so], check=True)
    f = ctypes.CDLL(so).bits
    f.restype = ctypes.c_uint32
    return f


def seen(i, len_, causal, window, sink, j):
    return 0 <= j < len_ and i >= 0 and (not causal or j <= i) and \
        (window <= 0 or i - j < window or j < sink)


WINDOWS = [0, 1, 31, 100, 1000, (1 << 30) - 1, 1 << 30, (1 << 31) - 129, (1 << 31) - 1]
SINKS = [0, 3, 33, 1 << 30, (1 << 31) - 1]


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("window", WINDOWS)
def test_bits_are_the_mask(bits, causal, window):
    rng = random.Random(window + causal)
    for len_ in (1, 33, 1000, 4096, 1 << 30):
        last = (len_ - 1) // 32 * 32
        for i in {0, 5, len_ // 2, len_ - 1, max(0, len_ - 100), -1, -40, -(1 << 30) + len_}:
            if i >= len_:
                continue
            for sink in SINKS:
                starts = {0, last, max(0, last - 32), max(0, i) // 32 * 32,
                          max(0, i - window) // 32 * 32, max(0, i - window + 32) // 32 * 32,
                          rng.randrange(0, last + 1) // 32 * 32}
                for k in starts:
                    if k > last:
                        continue
                    want = sum(1 << b for b in range(32) if seen(i, len_, causal, window, sink, k + b))
                    assert bits(i, len_, causal, window, sink, k) == want, (i, len_, sink, k)
