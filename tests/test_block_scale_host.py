"""Refusals of the block-scaled and cross calls on the host, before any CUDA call."""
import pytest

from paged_kv_cache_119_gb300 import _native as N
from paged_kv_cache_119_gb300 import build as B

FAKE = 1 << 24        # 16-byte-aligned non-null addresses, far apart; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def append_args(**kw):
    a = dict(k=FAKE, ks=1024, v=2 * FAKE, vs=1024, dtype=N.PA_BF16, kc=3 * FAKE, vc=4 * FAKE, ksc=5 * FAKE,
             vsc=6 * FAKE, stride=8, num_blocks=10, bt=7 * FAKE, bt_stride=8, cl=8 * FAKE, qs=9 * FAKE, T=3,
             mq=3, S=2, Hkv=8, D=128, B=16, stream=0)
    a.update(kw)
    return list(a.values())


BAD_APPEND = [
    (dict(dtype=7), N.PA_ERR_INVALID),
    (dict(dtype=N.PA_F32), N.PA_ERR_UNSUPPORTED),
    (dict(dtype=N.PA_FP8_E4M3), N.PA_ERR_INVALID),
    (dict(D=96), N.PA_ERR_UNSUPPORTED),
    (dict(B=8), N.PA_ERR_UNSUPPORTED),
    (dict(stride=7), N.PA_ERR_INVALID),                           # fewer scales than heads
    (dict(ks=1016), N.PA_ERR_INVALID),                            # shorter than a row
    (dict(vs=1028), N.PA_ERR_INVALID),                            # rows off 16 bytes
    (dict(k=FAKE + 8), N.PA_ERR_INVALID),
    (dict(ksc=5 * FAKE + 2), N.PA_ERR_INVALID),
    (dict(bt=7 * FAKE + 2), N.PA_ERR_INVALID),
    (dict(kc=0), N.PA_ERR_INVALID),
    (dict(vsc=0), N.PA_ERR_INVALID),
    (dict(qs=0), N.PA_ERR_INVALID),
    (dict(vc=3 * FAKE + 1024), N.PA_ERR_INVALID),                 # the pools overlap
    (dict(vsc=5 * FAKE + 64), N.PA_ERR_INVALID),                  # the scales overlap
    (dict(ksc=3 * FAKE), N.PA_ERR_INVALID),                       # scales inside a pool
    (dict(kc=FAKE), N.PA_ERR_INVALID),                            # a pool over k's rows
    (dict(ksc=8 * FAKE), N.PA_ERR_INVALID),                       # scales over the lengths
    (dict(T=-1), N.PA_ERR_INVALID),
    (dict(mq=-1), N.PA_ERR_INVALID),
    (dict(S=70000), N.PA_ERR_INVALID),
    (dict(num_blocks=0), N.PA_ERR_INVALID),
    (dict(num_blocks=1 << 28), N.PA_ERR_INVALID),                 # 2^31 cells
    (dict(bt_stride=1 << 28), N.PA_ERR_INVALID),                  # positions beyond 2^30
    (dict(T=0, k=0), N.PA_OK),
    (dict(S=0, kc=0), N.PA_OK),
    (dict(mq=0), N.PA_OK),
]


@pytest.mark.parametrize("kw,status", BAD_APPEND)
def test_append_rejects(lib, kw, status):
    assert lib.pa_append_fp8_block(*append_args(**kw)) == status


def rotary_args(**kw):
    freq = kw.pop("freq", [1.0] * 64)
    import ctypes
    buf = (ctypes.c_double * 64)(*freq)
    a = dict(qo=20 * FAKE, qos=4096, q=21 * FAKE, qs_=4096, k=FAKE, ks=1024, v=2 * FAKE, vs=1024,
             dtype=N.PA_BF16, kc=3 * FAKE, vc=4 * FAKE, ksc=5 * FAKE, vsc=6 * FAKE, stride=8, num_blocks=10,
             bt=7 * FAKE, bt_stride=8, cl=8 * FAKE, qs=9 * FAKE, pos=0, T=3, mq=3, S=2, Hq=32, Hkv=8, D=128,
             B=16, freq=ctypes.addressof(buf), rot=128, inter=0, mag=1.0, stream=0)
    a.update(kw)
    return list(a.values()), buf


@pytest.mark.parametrize("kw,status", BAD_APPEND[:-3] + [
    (dict(rot=0), N.PA_ERR_INVALID),
    (dict(rot=3), N.PA_ERR_INVALID),
    (dict(rot=130), N.PA_ERR_INVALID),
    (dict(freq=[2.0 ** 21] * 64), N.PA_ERR_INVALID),
    (dict(freq=[float("nan")] * 64), N.PA_ERR_INVALID),
    (dict(mag=float("inf")), N.PA_ERR_INVALID),
    (dict(q=0), N.PA_ERR_INVALID),
    (dict(qos=4088), N.PA_ERR_INVALID),
    (dict(qo=21 * FAKE + 16), N.PA_ERR_INVALID),                  # half over q
    (dict(qo=FAKE), N.PA_ERR_INVALID),                            # over k
    (dict(qo=3 * FAKE), N.PA_ERR_INVALID),                        # over a pool
    (dict(qo=9 * FAKE), N.PA_ERR_INVALID),                        # over query_start
    (dict(pos=3 * FAKE), N.PA_ERR_INVALID),                       # positions inside a pool
    (dict(pos=22 * FAKE + 2), N.PA_ERR_INVALID),
    (dict(T=0), N.PA_OK),
])
def test_rotary_append_rejects(lib, kw, status):
    args, keep = rotary_args(**kw)
    assert lib.pa_rotary_and_append_fp8_block(*args) == status


def attn_args(fn, **kw):
    decode = "decode" in fn
    a = dict(out=FAKE, out_dtype=N.PA_BF16, q=2 * FAKE)
    if fn == "pa_cross_attention":
        a.update(kc=3 * FAKE, vc=4 * FAKE, kv_dtype=N.PA_BF16)
    else:
        a.update(q_dtype=N.PA_BF16, kc=3 * FAKE, vc=4 * FAKE, ksc=5 * FAKE, vsc=6 * FAKE)
    if fn.endswith("block"):
        a.update(stride=4)
    a.update(num_blocks=10, bt=7 * FAKE, bt_stride=8, cl=8 * FAKE)
    if not decode:
        a.update(qs=9 * FAKE, rows=5, mq=4)
    a.update(max_ctx=64, S=2, Hq=8, Hkv=4, D=128, B=16, scale=0.1, part=0, ws=0, ws_bytes=0, stream=0)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


ALL = ["pa_decode_fp8_block", "pa_chunk_attention_fp8_block", "pa_cross_attention_fp8_block",
       "pa_cross_attention_fp8", "pa_cross_attention"]


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=N.PA_F16), N.PA_ERR_INVALID),
    (dict(Hq=9), N.PA_ERR_INVALID),
    (dict(D=96), N.PA_ERR_UNSUPPORTED),
    (dict(B=8), N.PA_ERR_UNSUPPORTED),
    (dict(max_ctx=129), N.PA_ERR_INVALID),
    (dict(max_ctx=-1), N.PA_ERR_INVALID),
    (dict(num_blocks=0), N.PA_ERR_INVALID),
    (dict(num_blocks=1 << 30), N.PA_ERR_INVALID),
    (dict(scale=float("inf")), N.PA_ERR_INVALID),
    (dict(part=64), N.PA_ERR_INVALID),
    (dict(q=0), N.PA_ERR_INVALID),
    (dict(q=2 * FAKE + 8), N.PA_ERR_INVALID),
    (dict(out=3 * FAKE), N.PA_ERR_INVALID),
    (dict(out=8 * FAKE), N.PA_ERR_INVALID),
    (dict(cl=8 * FAKE + 2), N.PA_ERR_INVALID),
    (dict(S=70000), N.PA_ERR_INVALID),
    (dict(S=0), N.PA_OK),
])
def test_attention_rejects(lib, fn, kw, status):
    assert getattr(lib, fn)(*attn_args(fn, **kw)) == status


@pytest.mark.parametrize("fn", ALL[:3])
@pytest.mark.parametrize("kw,status", [
    (dict(stride=3), N.PA_ERR_INVALID),
    (dict(stride=0), N.PA_ERR_INVALID),
    (dict(stride=-4), N.PA_ERR_INVALID),
    (dict(ksc=0), N.PA_ERR_INVALID),
    (dict(vsc=6 * FAKE + 2), N.PA_ERR_INVALID),
    (dict(out=5 * FAKE), N.PA_ERR_INVALID),                       # out over the scales
    (dict(q_dtype=N.PA_F32, out_dtype=N.PA_F32), N.PA_ERR_UNSUPPORTED),
])
def test_block_attention_rejects(lib, fn, kw, status):
    assert getattr(lib, fn)(*attn_args(fn, **kw)) == status


@pytest.mark.parametrize("fn", ALL)
def test_split_needs_a_workspace_apart_from_all(lib, fn):
    big = dict(max_ctx=1024, bt_stride=64, part=128)
    assert getattr(lib, fn)(*attn_args(fn, **big)) == N.PA_ERR_WORKSPACE
    rows = 2 if "decode" in fn else 5
    need = lib.pa_chunk_workspace_bytes(rows, 8, 128, 1024, 128)
    assert need > 0
    for at in (FAKE, 2 * FAKE, 3 * FAKE, 7 * FAKE, 8 * FAKE) + ((5 * FAKE,) if fn.endswith("block") else ()):
        assert getattr(lib, fn)(*attn_args(fn, **big, ws=at, ws_bytes=need)) == N.PA_ERR_INVALID


@pytest.mark.parametrize("fn", ALL[1:])
def test_row_arguments(lib, fn):
    for kw, status in [(dict(qs=0), N.PA_ERR_INVALID), (dict(rows=-1), N.PA_ERR_INVALID), (dict(rows=0), N.PA_OK),
                       (dict(mq=0), N.PA_OK), (dict(mq=-1), N.PA_ERR_INVALID), (dict(Hq=516), N.PA_ERR_INVALID)]:
        assert getattr(lib, fn)(*attn_args(fn, **kw)) == status, kw
    # a chunk is part of its context; rows across are as many as they are
    long = getattr(lib, fn)(*attn_args(fn, mq=65, out=3 * FAKE))
    assert long == N.PA_ERR_INVALID


def test_cross_of_one_byte_or_fp32_caches_has_its_own_name(lib):
    fn = "pa_cross_attention"
    assert lib.pa_cross_attention(*attn_args(fn, kv_dtype=N.PA_FP8_E4M3)) == N.PA_ERR_UNSUPPORTED
    assert lib.pa_cross_attention(*attn_args(fn, kv_dtype=N.PA_F32, out_dtype=N.PA_F32)) == N.PA_ERR_UNSUPPORTED
