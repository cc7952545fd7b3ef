"""Decode, chunk and cross attention over block-scaled E4M3 caches, and cross attention over the
other caches, against the definition in 64 bits.

Tolerance, derived: an fp32 dot of D <= 128 products with sum |q_i k_i| scale <= 16 is within
128 * 2^-24 * 16 = 1.2e-4 of the exact score, and x log2 e + log2 u, below 128 in magnitude, is
rounded to 2^-18: weights within e^(2 * 1.4e-4), so the output within 5.6e-4 sum p|v|.  P.V adds
2^-16 of it on the decode kernels and, on the tcgen05 chunk kernel, 2^-11 of it (one f16 term).
Weights are rounded relative to the largest p u of the row: each token may add 2^-24 of
448 max p u <= 448 * (the sum p|v| of a row can be that much below); the floor below covers it for
the contexts used here.  A native output is rounded once: eps / 2.
"""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
TOL = 5.6e-4 + 2.0 ** -11


def check(got, ref, size):
    assert torch.isfinite(got).all()
    err = np.abs(got.double().cpu().numpy() - ref)
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    floor = size.max(axis=-1, keepdims=True) * 2.0 ** -11
    tiny = 0.0 if got.dtype != torch.float16 else 2.0 ** -25      # half a step of f16's smallest
    limit = TOL * size + floor + half * (np.abs(ref) + TOL * size + floor) + tiny
    assert (err <= limit).all(), f"off by {float((err / limit).max()):.2f} of the tolerance"


def call(c, out=None, **kw):
    import paged_kv_cache_119_gb300 as pa
    out = torch.empty_like(c.q) if out is None else out
    if all(n == 1 for n in c.new) and c.causal:
        return pa.pa_decode_fp8_block(out, c.q, *c.args, c.scale, c.Hkv, c.B, **kw)
    fn = pa.pa_chunk_attention_fp8_block if c.causal else (
        pa.pa_cross_attention_fp8_block if c.scales and c.scales[0].dim() == 2 else
        pa.pa_cross_attention_fp8 if c.scales else pa.pa_cross_attention)
    kw.setdefault("max_query_len", max(c.new))
    return fn(out, c.q, *c.args, c.query_start, c.scale, c.Hkv, c.B, **kw)


def no_error():
    import paged_kv_cache_119_gb300 as pa
    torch.cuda.synchronize()
    return pa.pa_get_device_error() == 0


LENS = [1, 15, 16, 17, 130, 257, 600, 33]


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (9, 3), (8, 2), (8, 1), (14, 2), (24, 1), (64, 1), (5, 1)])
def test_decode(Hq, Hkv, D, B, dtype, pow2):
    c = R.build(21, LENS, [1] * len(LENS), Hq, Hkv, D, B, dtype, pow2=pow2, pad=Hkv != 3)
    ref, size = R.attend(c)
    for part in (0, -1, 128):
        out = torch.empty(c.q.shape, device="cuda") if part == 128 else None
        check(call(c, out, partition_size=part), ref, size)
    assert no_error()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("Hq,Hkv,new", [(4, 4, [2, 1, 3, 4]), (8, 2, [5, 2, 7, 1]), (8, 1, [3, 4, 1, 2]),
                                        (16, 2, [40, 3, 33, 64]), (7, 1, [65, 10, 1, 40]), (2, 2, [300, 1, 129, 0])])
def test_chunk(Hq, Hkv, new, D, B, dtype):
    lens = [n + extra for n, extra in zip(new, (90, 600, 0, 31))]
    c = R.build(22, lens, new, Hq, Hkv, D, B, dtype)
    ref, size = R.attend(c)
    for part in (0, -1, 128):
        check(call(c, partition_size=part), ref, size)
    assert no_error()


@pytest.mark.parametrize("kind", ["block", "head", "half"])
@pytest.mark.parametrize("D,B,dtype", [(128, 16, torch.bfloat16), (128, 32, torch.float16), (64, 32, torch.bfloat16),
                                       (64, 16, torch.float16)])
@pytest.mark.parametrize("Hq,Hkv,new", [(4, 4, [1, 1, 1, 1, 1]), (8, 2, [5, 2, 7, 1, 0]), (16, 2, [40, 3, 33, 64, 9]),
                                        (3, 1, [300, 1, 129, 65, 2])])
def test_cross(kind, Hq, Hkv, new, D, B, dtype):
    lens = [90, 17, 0, 700, 1]                    # fewer tokens than rows, none at all, one
    c = R.build(23, lens, new, Hq, Hkv, D, B, dtype, causal=False, kind=kind)
    ref, size = R.attend(c)
    for part in (0, -1, 128):
        got = call(c, torch.full(c.q.shape, float("nan"), device="cuda"), partition_size=part)
        check(got, ref, size)
        at = int(c.query_start[2])
        assert (got[at:at + new[2]] == 0).all()   # an empty context
    assert no_error()


@pytest.mark.parametrize("kind", ["block", "half"])
@pytest.mark.parametrize("rows", [1, 6, 200])
def test_cross_over_nothing(kind, rows):
    c = R.build(24, [0, 0], [rows, rows], 8, 2, 128, 16, torch.bfloat16, causal=False, kind=kind)
    for kw in (dict(), dict(max_context_len=0)):
        assert (call(c, torch.full(c.q.shape, float("nan"), device="cuda"), **kw) == 0).all()
    assert no_error()


def test_decode_of_an_empty_context():
    c = R.build(25, [0, 40, 0], [1, 1, 1], 8, 2, 128, 16, torch.float16)
    c.lens, c.new = [0, 40, 0], [1, 1, 1]
    got = call(c, torch.full(c.q.shape, float("nan"), device="cuda"))
    assert (got[0] == 0).all() and (got[2] == 0).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("Hq,Hkv,new,D", [(2, 2, 1, 128), (8, 1, 1, 128), (16, 1, 1, 128), (4, 2, 1, 64),
                                          (8, 1, 40, 128)])
def test_scales_far_apart(Hq, Hkv, new, D):
    """V scales over 2^-40 .. 2^40: what small blocks add is lost beside large ones of any weight,
    as it is in the sum itself, but a row's weights still sum to one."""
    c = R.build(26, [200, 90], [new, new], Hq, Hkv, D, 16, torch.float16, vscale=(-40, 40))
    ref, size = R.attend(c)
    check(call(c, torch.empty(c.q.shape, device="cuda")), ref, size)


@pytest.mark.parametrize("Hq,Hkv,new,D,B", [(2, 2, 1, 128, 16), (8, 1, 1, 128, 32), (16, 1, 1, 128, 16),
                                            (4, 2, 1, 64, 16), (8, 1, 40, 128, 16)])
@pytest.mark.parametrize("ends", [(2.0 ** -40, 2.0 ** 4), (2.0 ** -8, 2.0 ** 40)])
def test_weight_on_a_small_block(Hq, Hkv, new, D, B, ends):
    """The first block holds tiny values and nearly all the weight (a sink): the sum of weights
    keeps it whatever its scale is against the others'."""
    small, large = ends
    L = 4 * B + new
    c = R.build(27, [L], [new], Hq, Hkv, D, B, torch.float16)
    c.q.fill_(1.0)
    # keys: 1 in the first block (score D / sqrt(D)), 0 elsewhere; values: 1 code each
    k = torch.zeros(tuple(c.pools[0].shape), dtype=torch.uint8)
    k[int(c.table_np[0, 0])] = 0x38                # 1.0
    v = torch.full(tuple(c.pools[1].shape), 0x38, dtype=torch.uint8)
    c.pools[0].view(torch.uint8).copy_(k)
    c.pools[1].view(torch.uint8).copy_(v)
    c.scales[0].fill_(1.0)
    c.scales[1].fill_(large)
    c.scales[1][int(c.table_np[0, 0])] = small
    got = call(c, torch.empty(c.q.shape, device="cuda")).double().cpu()
    e = np.exp(D ** 0.5)
    for j in range(new):
        seen = L - new + j + 1
        want = (B * e * small + (seen - B) * large) / (B * e + (seen - B))
        assert abs(float(got[j].min()) / want - 1) <= TOL and abs(float(got[j].max()) / want - 1) <= TOL


def test_scales_beyond_the_bounds_count_as_the_bounds():
    c = R.build(28, [40], [1], 2, 2, 128, 16, torch.float16)
    blocks = [int(b) for b in c.table_np[0, :3]]
    outs = []
    for lo, hi in ((2.0 ** -48, 2.0 ** 48), (2.0 ** -60, 2.0 ** 90), (0.0, float("inf"))):
        for s in c.scales:
            s[blocks[0]], s[blocks[1]], s[blocks[2]] = lo, 2.0 ** -7, 2.0 ** -7
        c.scales[1][blocks[2]] = hi
        outs.append(call(c, torch.empty(c.q.shape, device="cuda")).clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bad_blocks_and_lengths():
    import paged_kv_cache_119_gb300 as pa
    from paged_kv_cache_119_gb300 import _native as N
    for Hq, Hkv, new, causal in [(2, 2, 1, True), (8, 1, 1, True), (16, 1, 1, True), (8, 1, 4, True), (8, 1, 40, True),
                                 (8, 1, 40, False), (2, 2, 3, False)]:
        c = R.build(29, [100, 200, 60], [new] * 3, Hq, Hkv, 128, 16, torch.bfloat16, causal=causal)
        good = call(c).clone()
        for bad in (-1, c.pools[0].shape[0], 2 ** 31 - 1):
            keep = int(c.table[1, 2])
            c.table[1, 2] = bad
            got = call(c)
            torch.cuda.synchronize()
            assert pa.pa_get_device_error() == N.PA_DEVERR_BLOCK_ID
            assert torch.equal(got[:new], good[:new]) and torch.equal(got[2 * new:], good[2 * new:])
            assert torch.isnan(got[new:2 * new]).all()
            c.table[1, 2] = keep
        for L in (-1, 10 ** 6) + ((new - 1,) if causal and new > 1 else ()):
            c.context_lens[1] = L
            got = call(c)
            torch.cuda.synchronize()
            assert pa.pa_get_device_error() == N.PA_DEVERR_CONTEXT_LEN
            assert torch.equal(got[:new], good[:new]) and torch.isnan(got[new:2 * new]).all()
        c.context_lens[1] = 200
        if new > 1:                                # rows that no sequence owns stay as they were
            out = torch.full(c.q.shape, 7.0, dtype=c.dtype, device="cuda")
            c.query_start[3] -= 1
            call(c, out)
            torch.cuda.synchronize()
            assert pa.pa_get_device_error() == N.PA_DEVERR_CONTEXT_LEN
            assert (out[-1] == 7).all()
        assert no_error()


def test_python_refusals():
    import paged_kv_cache_119_gb300 as pa
    c = R.build(30, [100, 200], [3, 3], 8, 2, 128, 16, torch.bfloat16)
    out = torch.empty_like(c.q)
    base = dict(out=out, q=c.q, k_cache=c.pools[0], v_cache=c.pools[1], k_scales=c.scales[0], v_scales=c.scales[1],
                block_tables=c.table, context_lens=c.context_lens, query_start=c.query_start, scale=c.scale,
                num_kv_heads=2, block_size=16, max_query_len=3)
    for kw, err in [(dict(k_scales=c.scales[0][:, :1]), ValueError), (dict(v_scales=c.scales[1].half()), ValueError),
                    (dict(v_scales=c.scales[1].cpu()), ValueError), (dict(q=c.q.float()), (TypeError, ValueError)),
                    (dict(k_cache=c.pools[0].float()), TypeError), (dict(query_start=c.context_lens), ValueError),
                    (dict(num_kv_heads=1), ValueError), (dict(block_tables=c.table.long()), TypeError)]:
        for fn in (pa.pa_chunk_attention_fp8_block, pa.pa_cross_attention_fp8_block):
            with pytest.raises(err):
                fn(**{**base, **kw})


def test_a_long_cache_beyond_two_to_the_31_bytes():
    """Cells past 2^31 bytes of the pools (a block's offset does not fit 32 bits)."""
    import paged_kv_cache_119_gb300 as pa
    H, D, B = 8, 128, 16
    N = (1 << 31) // (H * B * D) + 64
    k, v = (torch.zeros((N, H, B, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((N, H), device="cuda") for _ in range(2))
    table = torch.arange(N - 4, N, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn((50, 2 * H, D), device="cuda", generator=g).half()
    pa.pa_append_fp8_block(x[:, :H], x[:, H:], k, v, ks, vs, table, lens, start, max_query_len=50)
    c = R.Case()
    c.lens, c.new, c.Hq, c.Hkv, c.D, c.causal, c.scale = [50], [1], 2 * H, H, D, True, D ** -0.5
    ids = table[0].long()
    dense = [(p[ids].view(torch.float8_e4m3fn).double() * s[ids].double()[:, :, None, None]).transpose(0, 1)
             .reshape(H, -1, D)[:, :50].cpu() for p, s in ((k, ks), (v, vs))]
    c.K, c.V = [dense[0]], [dense[1]]
    assert (c.K[0] - x[:, :H].double().cpu().transpose(0, 1)).abs().max() < 0.2
    c.q = torch.randn((1, 2 * H, D), device="cuda", generator=g).half()
    ref, size = R.attend(c)
    out = torch.empty_like(c.q)
    check(pa.pa_decode_fp8_block(out, c.q, k, v, ks, vs, table, lens, c.scale, H, B), ref, size)


def test_a_bound_that_changes_between_calls():
    """max_context_len is taken by its value at each call: the same object, holding another number
    the second time (the first call's contexts fit in 16 tokens, the second's do not)."""
    bound = torch.tensor(16)
    c = R.build(40, [90, 64], [1, 1], 8, 2, 128, 16, torch.bfloat16)
    ref, size = R.attend(c)
    whole = c.context_lens.clone()
    c.context_lens.fill_(16)
    call(c, max_context_len=bound)
    bound.fill_(90)
    c.context_lens.copy_(whole)
    check(call(c, max_context_len=bound), ref, size)
    assert no_error()
