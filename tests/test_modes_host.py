"""Refusals of the modified-score and shared-prefix calls at the C interface (no GPU: every
call here returns before it launches anything, and the pointers are never followed)."""
import pytest

from paged_kv_cache_119_gb300 import _native as N


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_119_gb300 import build as b
    b.build()
    return N.load()


FAKE = 1 << 28
INV, UNS, WS = N.PA_ERR_INVALID, N.PA_ERR_UNSUPPORTED, N.PA_ERR_WORKSPACE


def decode_args(**kw):
    a = dict(out=FAKE, out_dtype=N.PA_BF16, q=FAKE * 2, k_cache=FAKE * 3, v_cache=FAKE * 4,
             kv_dtype=N.PA_BF16, num_blocks=100, table=FAKE * 5, stride=40, lens=FAKE * 6,
             max_context=640, S=3, Hq=8, Hkv=2, D=128, B=16, scale=0.1, cap=0.0, slopes=0, window=0,
             glob=0, max_glob=0, part=0, ws=0, ws_bytes=0, stream=0)
    a.update(kw)
    return a


DECODE = [
    (dict(kv_dtype=77), INV),
    (dict(kv_dtype=N.PA_FP8_E4M3), INV),                     # has its own call
    (dict(out_dtype=N.PA_F16), INV),                         # neither fp32 nor the query type
    (dict(S=-1), INV), (dict(S=65536), INV),
    (dict(Hkv=0), INV), (dict(Hq=7), INV),
    (dict(D=80), UNS), (dict(B=8), UNS),
    (dict(num_blocks=0), INV), (dict(num_blocks=1 << 31), INV),
    (dict(num_blocks=1 << 30), INV),                         # x 2 heads: tile index beyond 32 bits
    (dict(stride=0), INV), (dict(max_context=641), INV),     # longer than the table's row
    (dict(max_context=-1), INV),
    (dict(max_context=(1 << 30) + 1, stride=1 << 27), INV),
    (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(cap=-1.0), INV), (dict(cap=float("nan")), INV), (dict(cap=float("inf")), INV),
    (dict(cap=1e-31), INV),
    (dict(window=-1), INV), (dict(glob=FAKE * 7, max_glob=-1), INV),
    (dict(part=64), INV),
    (dict(out=0), INV), (dict(q=0), INV), (dict(k_cache=0), INV), (dict(table=0), INV), (dict(lens=0), INV),
    (dict(q=FAKE * 2 + 8), INV), (dict(slopes=FAKE * 7 + 2), INV),
    (dict(out=FAKE * 2 + 64), INV),                          # out over q
    (dict(out=FAKE * 3), INV), (dict(glob=FAKE, max_glob=3), INV), (dict(slopes=FAKE), INV),
    (dict(part=128), WS),                                    # a split without a workspace
    (dict(part=128, ws=FAKE * 8, ws_bytes=100), WS),
    (dict(part=128, ws=FAKE * 8 + 4, ws_bytes=1 << 20), WS),
    (dict(part=128, ws=FAKE * 2, ws_bytes=1 << 20), INV),    # the workspace over q
    (dict(part=128, ws=FAKE, ws_bytes=1 << 20), INV),        # and over out
    (dict(S=0), N.PA_OK),
]


@pytest.mark.parametrize("kw,status", DECODE, ids=str)
def test_decode_mod_rejects(lib, kw, status):
    assert lib.pa_decode_mod(*decode_args(**kw).values()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q_dtype=N.PA_F32, out_dtype=N.PA_F32), UNS), (dict(k_scale=0), INV), (dict(v_scale=0), INV),
    (dict(q_dtype=N.PA_FP8_E4M3), INV), (dict(cap=-2.0), INV), (dict(S=0), N.PA_OK)], ids=str)
def test_decode_mod_fp8_rejects(lib, kw, status):
    a = decode_args()
    names = [n for n in a if n != "kv_dtype"]
    names.insert(names.index("q") + 1, "q_dtype")
    names[names.index("v_cache") + 1:names.index("v_cache") + 1] = ["k_scale", "v_scale"]
    a = {**a, "q_dtype": N.PA_BF16, "k_scale": FAKE * 9, "v_scale": FAKE * 10, **kw}
    assert lib.pa_decode_mod_fp8(*[a[n] for n in names]) == status


def chunk_args(**kw):
    a = dict(out=FAKE, out_dtype=N.PA_BF16, q=FAKE * 2, k_cache=FAKE * 3, v_cache=FAKE * 4,
             kv_dtype=N.PA_BF16, num_blocks=100, table=FAKE * 5, stride=40, lens=FAKE * 6, start=FAKE * 7,
             tokens=30, max_query=20, max_context=640, S=3, Hq=8, Hkv=2, D=128, B=16, scale=0.1, cap=0.0,
             slopes=0, window=0, glob=0, max_glob=0, part=0, ws=0, ws_bytes=0, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(kv_dtype=N.PA_F32, out_dtype=N.PA_F32), UNS), (dict(kv_dtype=N.PA_FP8_E4M3), UNS),
    (dict(Hq=258, Hkv=2), INV),                              # more than 128 heads a kv head
    (dict(max_query=641), INV), (dict(max_query=-1), INV), (dict(tokens=-1), INV),
    (dict(tokens=1 << 31), INV), (dict(start=0), INV), (dict(window=-5), INV), (dict(cap=1e31), INV),
    (dict(part=128), WS), (dict(part=128, ws=FAKE * 2, ws_bytes=1 << 24), INV),
    (dict(start=FAKE), INV),                                 # out over query_start
    # the kv heads times the row tiles are a grid dimension
    (dict(max_query=1 << 29, max_context=1 << 29, stride=1 << 25, S=1), INV),
    # partitions times row tiles beyond a grid (256 rows of 65536 parts, 2 heads, 3000 sequences)
    (dict(max_query=4096, max_context=1 << 23, stride=1 << 19, S=3000, part=128, tokens=1, Hq=16,
          ws=FAKE * 64, ws_bytes=1 << 40), INV),
    (dict(tokens=0), N.PA_OK), (dict(S=0), N.PA_OK), (dict(max_query=0), N.PA_OK)], ids=str)
def test_chunk_mod_rejects(lib, kw, status):
    assert lib.pa_chunk_attention_mod(*chunk_args(**kw).values()) == status


def prefix_args(**kw):
    a = dict(out=FAKE, out_dtype=N.PA_BF16, q=FAKE * 2, k_cache=FAKE * 3, v_cache=FAKE * 4,
             kv_dtype=N.PA_BF16, num_blocks=100, table=FAKE * 5, stride=40, lens=FAKE * 6, plens=FAKE * 7,
             start=FAKE * 8, groups=2, max_group=2, max_prefix=320, max_suffix=320, S=3, Hq=8, Hkv=2,
             D=128, B=16, scale=0.1, part=0, ws=FAKE * 9, ws_bytes=1 << 24, stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(kv_dtype=N.PA_F32, out_dtype=N.PA_F32), UNS), (dict(kv_dtype=N.PA_FP8_E4M3), UNS),
    (dict(Hq=258), INV), (dict(S=65535, max_group=9), INV), (dict(D=96), UNS),
    (dict(max_prefix=-16), INV), (dict(max_suffix=-1), INV),
    (dict(max_prefix=312), INV),                             # no whole number of blocks
    (dict(max_prefix=656), INV),                             # longer than the table's row
    (dict(max_prefix=1 << 30, stride=1 << 26), INV),         # with the suffix beyond 2^30
    (dict(groups=0), INV), (dict(groups=4), INV), (dict(max_group=0), INV), (dict(max_group=4), INV),
    (dict(plens=0), INV), (dict(start=0), INV), (dict(q=0), INV), (dict(k_cache=FAKE * 3 + 4), INV),
    (dict(part=96), INV),
    (dict(ws=0), WS), (dict(ws_bytes=64), WS), (dict(ws=FAKE * 9 + 8), WS),
    (dict(ws=FAKE), INV), (dict(ws=FAKE * 7), INV), (dict(out=FAKE * 8), INV), (dict(out=FAKE * 4), INV),
    (dict(S=0, groups=0, max_group=0), N.PA_OK)], ids=str)
def test_prefix_rejects(lib, kw, status):
    assert lib.pa_decode_prefix(*prefix_args(**kw).values()) == status


def test_prefix_workspace(lib):
    f = lib.pa_decode_prefix_workspace_bytes
    assert f(-1, 8, 128, 64, 64, 0) == 0 and f(4, 8, 128, -1, 64, 0) == 0
    row = 4 * (128 + 2)
    assert f(4, 8, 128, 1024, 512, -1) == 4 * 8 * 2 * row                # a part of each pass
    assert f(4, 8, 128, 1024, 512, 128) == 4 * 8 * 12 * row
    assert f(4, 8, 128, 1024, 513, 0) == 4 * 8 * 4 * row                 # parts of 512 at least


def test_the_binding_refuses_host_tensors():
    import torch

    import paged_kv_cache_119_gb300 as P
    q, pool = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        P.pa_decode_mod(q, q, pool, pool, table, lens, 0.1, 2, 16)
    with pytest.raises(ValueError):
        P.pa_decode_prefix(q, q, pool, pool, table, lens, lens, lens, 0.1, 2, 16, max_group_size=1, max_prefix_len=0)
    with pytest.raises(ValueError):
        P.pa_rotary_and_cache(q, q, q, q, pool, pool, lens.long(), lens, [0.1] * 32)


@pytest.mark.parametrize("name", ["table", "lens", "slopes", "glob"])
def test_decode_mod_rejects_unaligned_arrays(lib, name):
    a = decode_args(slopes=FAKE * 11, glob=FAKE * 12, max_glob=4)
    a[name] += 2
    assert lib.pa_decode_mod(*a.values()) == INV


@pytest.mark.parametrize("name", ["table", "lens", "plens", "start"])
def test_prefix_rejects_unaligned_arrays(lib, name):
    a = prefix_args()
    a[name] += 2
    assert lib.pa_decode_prefix(*a.values()) == INV


def test_chunk_mod_rejects_an_unaligned_query_start(lib):
    assert lib.pa_chunk_attention_mod(*chunk_args(start=FAKE * 7 + 2).values()) == INV
