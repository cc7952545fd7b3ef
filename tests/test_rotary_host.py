"""The rotary entry points without a GPU: the frequency helper against its formulas, and
the refusals of the C ABI (nothing is launched, no pointer is read but inv_freq)."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_119_gb300 as P
from paged_kv_cache_119_gb300 import _native as N
from paged_kv_cache_119_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


@pytest.mark.parametrize("dim", [2, 4, 36, 64, 128, 256])
def test_frequencies_against_the_formulas(lib, dim):
    i = np.arange(dim // 2)
    f = 10000.0 ** (-2.0 * i / dim)
    # pow and one or two products in double: a few units of 2^-53
    np.testing.assert_allclose(P.pa_rotary_frequencies(dim), f, rtol=1e-14)
    np.testing.assert_allclose(P.pa_rotary_frequencies(dim, scaling="linear", factor=4.0), f / 4, rtol=1e-14)
    if dim >= 4:
        base = 500000.0 * 8.0 ** (dim / (dim - 2))
        got = P.pa_rotary_frequencies(dim, base=500000.0, scaling="ntk", factor=8.0)
        np.testing.assert_allclose(got, base ** (-2.0 * i / dim), rtol=1e-13)
        # the slowest pair ends exactly `factor` times slower
        np.testing.assert_allclose(got[-1], 500000.0 ** (-2.0 * (dim // 2 - 1) / dim) / 8.0, rtol=1e-13)
    got = P.pa_rotary_frequencies(dim, scaling="by_parts", factor=8.0, low_turns=1.0, high_turns=32.0,
                                  original_len=4096)
    turns = 4096 * f / (2 * math.pi)
    g = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
    np.testing.assert_allclose(got, g * f + (1 - g) * f / 8.0, rtol=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(base=1.0), dict(base=float("inf")),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
    dict(rotary_dim=2, scaling="ntk", factor=2.0), dict(scaling="by_parts", factor=2.0),
    dict(scaling="by_parts", factor=2.0, original_len=4096, low_turns=4.0, high_turns=4.0),
    dict(scaling="by_parts", factor=2.0, original_len=4096, low_turns=-1.0),
])
def test_frequencies_refuse(lib, kw):
    with pytest.raises(RuntimeError):
        P.pa_rotary_frequencies(**{**dict(rotary_dim=64), **kw})


def test_unknown_scaling_name():
    with pytest.raises(ValueError):
        P.pa_rotary_frequencies(64, scaling="other")


FAKE = 1 << 24
FREQ = (ctypes.c_double * 64)(*[0.5] * 64)
BIG = (ctypes.c_double * 64)(*[2.0 ** 20] * 64)


def rotary_args(**kw):
    a = dict(q_out=FAKE, q_out_stride=512, q=FAKE * 2, q_stride=512, k=FAKE * 3, k_stride=256, v=FAKE * 4,
             v_stride=256, dtype=N.PA_BF16, k_cache=FAKE * 5, v_cache=FAKE * 6, slots=FAKE * 7,
             positions=FAKE * 8, tokens=3, Hq=4, Hkv=2, D=128, B=16, num_blocks=10, freq=FREQ, rot=128,
             inter=0, magnitude=1.0, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=N.PA_FP8_E4M3), N.PA_ERR_INVALID),
    (dict(tokens=-1), N.PA_ERR_INVALID),
    (dict(Hq=0), N.PA_ERR_INVALID),
    (dict(num_blocks=0), N.PA_ERR_INVALID),
    (dict(rot=0), N.PA_ERR_INVALID),
    (dict(rot=63), N.PA_ERR_INVALID),
    (dict(rot=130), N.PA_ERR_INVALID),                       # beyond head_dim
    (dict(freq=None), N.PA_ERR_INVALID),
    (dict(freq=BIG), N.PA_ERR_INVALID),
    (dict(magnitude=float("nan")), N.PA_ERR_INVALID),
    (dict(D=4, rot=4, q_out_stride=16, q_stride=16, k_stride=8, v_stride=8), N.PA_ERR_UNSUPPORTED),
    (dict(q_stride=511), N.PA_ERR_INVALID),                  # not a whole 16-byte vector
    (dict(q_stride=504), N.PA_ERR_INVALID),                  # shorter than a row
    (dict(k=FAKE * 3 + 8), N.PA_ERR_INVALID),                # misaligned
    (dict(q=0), N.PA_ERR_INVALID),
    (dict(positions=0), N.PA_ERR_INVALID),
    (dict(q_out=FAKE * 2 + 512), N.PA_ERR_INVALID),          # q_out shifted against q
    (dict(q_out=FAKE * 2, q_out_stride=1024), N.PA_ERR_INVALID),   # in place, another stride
    (dict(q_out=FAKE * 3), N.PA_ERR_INVALID),                # q_out is k
    (dict(q_out=FAKE * 5), N.PA_ERR_INVALID),                # q_out in the cache
    (dict(v_cache=FAKE * 5 + 1024), N.PA_ERR_INVALID),       # caches overlap
    # views of one projection: rows of 4 q + 2 k + 2 v heads; q_out on top of k's part
    (dict(q=FAKE, q_stride=1024, k=FAKE + 1024, k_stride=1024, v=FAKE + 1536, v_stride=1024,
          q_out=FAKE + 512, q_out_stride=1024), N.PA_ERR_INVALID),
])
def test_rotary_rejects(lib, kw, status):
    assert lib.pa_rotary_and_cache(*rotary_args(**kw).values()) == status


def test_rotary_fp8_rejects(lib):
    a = rotary_args()
    names = list(a)
    cut = names.index("v_cache") + 1

    def call(ks, vs, **kw):
        b = list(rotary_args(**kw).values())
        return lib.pa_rotary_and_cache_fp8(*b[:cut], ks, vs, *b[cut:])

    assert call(0, FAKE * 9) == N.PA_ERR_INVALID
    assert call(FAKE * 9, 0) == N.PA_ERR_INVALID
    assert call(FAKE * 9, FAKE * 10, D=24, rot=24, q_out_stride=96, q_stride=96, k_stride=48,
                v_stride=48) == N.PA_ERR_UNSUPPORTED
    assert call(FAKE * 9, FAKE * 10, tokens=0) == N.PA_OK    # nothing to do, no launch


@pytest.mark.parametrize("kw", [dict(slots=FAKE * 7 + 4), dict(positions=FAKE * 8 + 2)])
def test_rotary_rejects_unaligned_arrays(lib, kw):
    assert lib.pa_rotary_and_cache(*rotary_args(**kw).values()) == N.PA_ERR_INVALID
