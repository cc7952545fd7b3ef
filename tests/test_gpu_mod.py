"""Attention with modified scores (pa_decode_mod, pa_chunk_attention_mod and their E4M3
forms) on the GPU against a plain 64-bit reference: tolerances are derived in
attn_reference.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import CHUNK_TOL, ROWS_TOL, build, check, reference

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_119_gb300 import build as b
    b.build()


@pytest.fixture(autouse=True)
def clear_error_word(built):
    P.pa_get_device_error()
    yield


def slopes_for(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


def run(c, decode, softcap=0.0, slopes=None, out_dtype=torch.float32, partition_size=0, max_global=None,
        scale=None, max_context_len=None, stream=None, workspace=None):
    out = torch.full(c.q.shape, float("nan"), dtype=out_dtype, device="cuda")
    kw = dict(softcap=softcap, alibi_slopes=slopes, window=c.window, global_lens=c.global_lens,
              max_global_len=max_global, partition_size=partition_size,
              max_context_len=max(c.lens) if max_context_len is None else max_context_len,
              stream=stream, workspace=workspace)
    scale = c.scale if scale is None else scale
    if decode:
        f = P.pa_decode_mod_fp8 if c.fp8 else P.pa_decode_mod
        f(out, c.q, *c.pools, c.table, c.context_lens, scale, c.Hkv, c.B, **kw)
    else:
        f = P.pa_chunk_attention_mod_fp8 if c.fp8 else P.pa_chunk_attention_mod
        f(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, scale, c.Hkv, c.B,
          max_query_len=max(c.new), **kw)
    torch.cuda.synchronize()
    return out


def compare(c, decode, tol, softcap=0.0, slopes=None, **kw):
    out = run(c, decode, softcap, slopes, **kw)
    assert P.pa_get_device_error() == 0
    ref, vmax = reference(c, softcap, slopes, scale=kw.get("scale"))
    check(out, ref, vmax, tol)
    return out


LENS = [1, 0, 15, 16, 17, 33, 130, 300, 777]
MODS = [dict(), dict(window=1), dict(window=16), dict(window=37), dict(window=500),
        dict(window=37, glob=5), dict(window=100, glob=64), dict(window=1, glob=1), dict(glob=40)]


@pytest.mark.parametrize("mods", MODS, ids=str)
@pytest.mark.parametrize("Hq,Hkv,D,B,dtype,fp8", [
    (4, 4, 128, 16, torch.float16, False), (6, 2, 64, 32, torch.bfloat16, False),
    (8, 2, 128, 16, torch.bfloat16, False), (8, 1, 128, 32, torch.float16, False),
    (14, 2, 128, 16, torch.bfloat16, False), (24, 2, 64, 16, torch.float16, False),
    (40, 1, 128, 16, torch.float16, False), (30, 1, 128, 16, torch.bfloat16, True),
    (3, 3, 64, 16, torch.float32, False), (8, 1, 128, 32, torch.float32, False),
    (2, 2, 128, 16, torch.bfloat16, True), (4, 2, 128, 32, torch.float16, True),
    (6, 2, 128, 16, torch.bfloat16, True), (8, 2, 128, 16, torch.float16, True),
    (8, 1, 128, 16, torch.bfloat16, True), (10, 2, 128, 32, torch.float16, True),
    (2, 2, 64, 16, torch.float16, True), (8, 2, 64, 32, torch.bfloat16, True),
    (8, 1, 64, 16, torch.bfloat16, True)])
def test_decode(Hq, Hkv, D, B, dtype, fp8, mods):
    glob = [mods["glob"]] * len(LENS) if "glob" in mods else None
    c = build(Hq + D + B, LENS, [1] * len(LENS), Hq, Hkv, D, B, dtype, fp8, mods.get("window", 0), glob)
    for part in (0, 128):
        compare(c, True, ROWS_TOL, softcap=3.0, slopes=slopes_for(Hq), partition_size=part)
        compare(c, True, ROWS_TOL, partition_size=part, max_global=mods.get("glob"))


@pytest.mark.parametrize("softcap", [0.0, 0.01, 1.0, 30.0, 1e6])
@pytest.mark.parametrize("Hq,fp8,dtype", [(2, False, torch.float32), (2, False, torch.float16),
                                          (8, False, torch.bfloat16), (4, True, torch.bfloat16)])
def test_caps(softcap, Hq, fp8, dtype):
    """Caps far below, near and far above the scores (the last is no cap to speak of)."""
    c = build(5, [200, 64], [1, 1], Hq, 2 if Hq > 2 else 1, 128, 16, dtype, fp8)
    compare(c, True, ROWS_TOL, softcap=softcap)
    compare(c, True, ROWS_TOL, softcap=softcap, scale=-0.05)
    compare(c, True, ROWS_TOL, softcap=softcap, scale=0.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq", [2, 8])
def test_native_outputs(dtype, Hq):
    c = build(6, LENS, [1] * len(LENS), Hq, 2, 128, 16, dtype, window=50, glob=[3] * len(LENS))
    compare(c, True, ROWS_TOL, softcap=20.0, out_dtype=dtype)


def test_many_sequences_of_one_head():
    """More CTAs than one wave: the longest-first order of the CUDA-core kernel."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 120, 300)]
    c = build(7, lens, [1] * 300, 16, 16, 64, 16, torch.float16)
    compare(c, True, ROWS_TOL, slopes=slopes_for(16))


@pytest.mark.parametrize("Hq,Hkv,fp8,dtype", [(2, 2, False, torch.float16), (8, 1, False, torch.bfloat16),
                                              (4, 1, True, torch.float16), (8, 1, True, torch.bfloat16)])
def test_long_context_automatic_split(Hq, Hkv, fp8, dtype):
    """Few sequences, long contexts: the automatic split, with and without a window."""
    lens = [9000, 4097, 1]
    for window, glob in ((0, None), (3000, [100, 1, 50])):
        c = build(8, lens, [1] * 3, Hq, Hkv, 128, 16, dtype, fp8, window, glob)
        compare(c, True, ROWS_TOL, softcap=50.0, max_global=100 if glob else None)


def test_global_lens_are_clamped():
    """Entries below 0, beyond the context and beyond max_global_len."""
    lens = [100, 100, 40]
    c = build(9, lens, [1] * 3, 4, 1, 128, 16, torch.bfloat16, window=10, glob=[-7, 20, 999])
    out = run(c, True, max_global=20)
    c2 = build(9, lens, [1] * 3, 4, 1, 128, 16, torch.bfloat16, window=10, glob=[0, 20, 20])
    assert torch.equal(c2.q, c.q)
    check(out, *reference(c2), ROWS_TOL)
    assert P.pa_get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,fp8,dtype", [
    (2, 2, 128, False, torch.float16), (4, 1, 64, False, torch.bfloat16), (8, 1, 128, False, torch.float16),
    (2, 1, 128, True, torch.bfloat16), (8, 1, 128, True, torch.float16), (2, 1, 64, True, torch.float16),
    (3, 1, 64, False, torch.float32)])
@pytest.mark.parametrize("window,glob", [(1, 0), (7, 0), (16, 16), (45, 3), (64, 17), (0, 0)])
def test_exactly_the_visible_tokens_count(Hq, Hkv, D, fp8, dtype, window, glob):
    """Equal scores: the output is the mean of the visible rows of V, so that one token too
    many or too few is off by 1 / n.  Equal weights are exact and V enters exactly; the sums
    of n terms round (or, on the tensor cores, truncate) in fp32: n 2^-23 max |v|."""
    lens = [97, 64, 33, 200]
    c = build(10, lens, [1] * 4, Hq, Hkv, D, 16, dtype, fp8, window, [glob] * 4 if glob else None, kstd=0.0)
    ref, vmax = reference(c)
    for part in (0, 128):
        out = run(c, True, partition_size=part)
        err = np.abs(out.double().cpu().numpy() - ref).max()
        assert err <= 220 * 2.0 ** -23 * vmax, err


# ------------------------------------------------------------------------------- chunks

CHUNKS = [(lens, new) for lens, new in [
    ([1, 40, 9, 0, 200, 333], [1, 3, 0, 0, 5, 2]),              # a few rows per kv head
    ([70, 129, 300, 64, 513], [70, 20, 100, 1, 77])]]           # long chunks


@pytest.mark.parametrize("mods", [dict(), dict(window=1), dict(window=50), dict(window=100, glob=30),
                                  dict(glob=60), dict(glob=300), dict(window=16, glob=64)], ids=str)
@pytest.mark.parametrize("shape", [0, 1], ids=["few", "long"])
@pytest.mark.parametrize("Hq,Hkv,D,B,dtype,fp8", [
    (4, 4, 128, 16, torch.float16, False), (8, 2, 128, 32, torch.bfloat16, False),
    (8, 1, 64, 16, torch.bfloat16, False), (5, 1, 64, 32, torch.float16, False),
    (4, 2, 128, 16, torch.bfloat16, True), (8, 1, 128, 32, torch.float16, True),
    (1, 1, 128, 16, torch.float16, True), (4, 1, 64, 16, torch.bfloat16, True)])
def test_chunk(Hq, Hkv, D, B, dtype, fp8, shape, mods):
    lens, new = CHUNKS[shape]
    glob = [mods["glob"]] * len(lens) if "glob" in mods else None
    c = build(11 + shape, lens, new, Hq, Hkv, D, B, dtype, fp8, mods.get("window", 0), glob)
    for part in (0, 128):
        compare(c, False, CHUNK_TOL, softcap=3.0, slopes=slopes_for(Hq), partition_size=part)
        compare(c, False, CHUNK_TOL, partition_size=part)


@pytest.mark.parametrize("Hq,D,fp8,dtype", [(4, 128, False, torch.float16), (4, 128, False, torch.bfloat16),
                                            (4, 64, False, torch.bfloat16), (4, 128, True, torch.float16)])
@pytest.mark.parametrize("window,glob", [(1, 0), (30, 0), (64, 10), (100, 129), (0, 90)])
def test_chunk_counts_exactly_the_visible_tokens(Hq, D, fp8, dtype, window, glob):
    """Equal scores, as for the decode: equal weights are exact in f16, bf16 V is exact in
    f16 for 2^-14 <= |v| (smaller values lose at most 2^-25)."""
    lens, new = [300, 130], [90, 130]
    c = build(12, lens, new, Hq, 1, D, 16, dtype, fp8, window, [glob] * 2 if glob else None, kstd=0.0)
    ref, vmax = reference(c)
    for part in (0, 128):
        out = run(c, False, partition_size=part)
        err = np.abs(out.double().cpu().numpy() - ref).max()
        assert err <= 320 * 2.0 ** -23 * vmax + 2.0 ** -25, err


def test_chunk_long_window_automatic_split():
    for fp8 in (False, True):
        c = build(13, [6000, 2500], [200, 64], 8, 1, 128, 16, torch.bfloat16, fp8, 1500, [64, 64])
        compare(c, False, CHUNK_TOL, softcap=30.0)


@pytest.mark.parametrize("mods", [dict(), dict(window=600, glob=100)], ids=str)
@pytest.mark.parametrize("dtype,fp8", [(torch.float16, False), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_chunk_last_wave_is_cut(dtype, fp8, mods):
    """168 units of one CTA each on 152 SMs: the last ones are split and merged, the others
    write their rows themselves; an empty chunk and a short context among the split ones."""
    lens = [1100 + 3 * i for i in range(17)] + [1300, 40, 1250, 1030]
    new = [40 - i % 3 for i in range(17)] + [40, 40, 0, 37]
    glob = [mods["glob"]] * len(lens) if "glob" in mods else None
    c = build(21, lens, new, 8, 8, 128, 16, dtype, fp8, mods.get("window", 0), glob)
    compare(c, False, CHUNK_TOL, softcap=30.0, max_global=mods.get("glob"))
    compare(c, False, CHUNK_TOL, slopes=slopes_for(8), max_global=mods.get("glob"))


@pytest.mark.parametrize("softcap", [0.01, 5.0, 1e6])
def test_chunk_caps_and_scales(softcap):
    for fp8 in (False, True):
        c = build(14, [150], [60], 8, 1, 128, 16, torch.bfloat16, fp8)
        for scale in (None, -0.05, 0.0):
            compare(c, False, CHUNK_TOL, softcap=softcap, scale=scale)


# ------------------------------------------------------- agreement with the plain calls

@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 2), (32, 8)])
def test_without_modifiers_it_is_the_plain_call(Hq, Hkv):
    c = build(15, LENS, [1] * len(LENS), Hq, Hkv, 128, 16, torch.bfloat16)
    a = run(c, True)
    b = torch.empty_like(a)
    P.pa_decode(b, c.q, *c.pools, c.table, c.context_lens, c.scale, c.Hkv, c.B)
    assert (a - b).abs().max() <= 1e-4      # two fp32 evaluations, each far inside this


# ------------------------------------------------------------------ errors and refusals

def test_errors_are_flagged_and_poison_only_their_rows():
    c = build(16, [100, 60, 90], [1] * 3, 8, 2, 128, 16, torch.float16, window=20)
    good = run(c, True)
    c.context_lens[1] = -3
    out = run(c, True)
    assert P.pa_get_device_error() == 2
    assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c.context_lens[1] = 60
    c.table[2, 90 // 16] = 10 ** 6          # a block the window sees
    out = run(c, True)
    assert P.pa_get_device_error() == 1
    assert torch.isnan(out[2]).all() and torch.equal(out[0], good[0]) and torch.equal(out[1], good[1])
    # split: the merge carries the poison
    c = build(16, [300, 260, 290], [1] * 3, 8, 2, 128, 16, torch.float16)
    c.table[2, 9] = -1
    out = run(c, True, partition_size=128)
    assert P.pa_get_device_error() == 1
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all()


def test_chunk_errors():
    c = build(17, [100, 200], [40, 50], 8, 2, 128, 16, torch.bfloat16, window=30)
    good = run(c, False)
    c.context_lens[0] = 39                  # fewer tokens than rows
    for part in (0, 128):
        out = run(c, False, partition_size=part)
        assert P.pa_get_device_error() & 2
        assert torch.isnan(out[:40]).all()
        assert (out[40:] - good[40:]).abs().max() <= 1e-2


def test_rows_behind_the_last_sequence_stay():
    """Rows that no sequence owns keep what they hold, and are flagged."""
    c = build(18, [50, 80], [10, 20], 4, 1, 128, 16, torch.float16)
    c.query_start[2] = 25
    out = torch.full(c.q.shape, 7.0, dtype=torch.float32, device="cuda")
    P.pa_chunk_attention_mod(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, c.scale, 1, 16,
                             max_query_len=20, window=9, partition_size=-1)
    torch.cuda.synchronize()
    assert (out[25:] == 7.0).all() and torch.isfinite(out[:25]).all()
    assert P.pa_get_device_error() == 2


def test_refusals():
    c = build(19, [50, 80], [1, 1], 4, 2, 128, 16, torch.float16)
    out = torch.empty(c.q.shape, device="cuda")
    args = (out, c.q, *c.pools, c.table, c.context_lens, c.scale, 2, 16)
    for kw in (dict(softcap=-1.0), dict(softcap=float("inf")), dict(softcap=float("nan")),
               dict(softcap=1e-35), dict(window=-1), dict(partition_size=64), dict(max_context_len=10 ** 6),
               dict(global_lens=c.context_lens, max_global_len=-1)):
        with pytest.raises(RuntimeError):
            P.pa_decode_mod(*args, **kw)
    for kw in (dict(alibi_slopes=torch.ones(3, device="cuda")),
               dict(alibi_slopes=torch.ones(4, device="cuda").double()),
               dict(global_lens=c.context_lens[:1])):
        with pytest.raises(ValueError):
            P.pa_decode_mod(*args, **kw)
    with pytest.raises(TypeError):
        P.pa_decode_mod(*args, global_lens=c.context_lens.long())
    f32 = build(19, [50], [3], 4, 2, 128, 16, torch.float32)
    with pytest.raises(RuntimeError):
        P.pa_chunk_attention_mod(torch.empty_like(f32.q), f32.q, *f32.pools, f32.table, f32.context_lens,
                                 f32.query_start, f32.scale, 2, 16, max_query_len=3)


# ------------------------------------------------------------------- streams and graphs

def test_captured_and_replayed_on_another_stream():
    """A captured call replays on new lengths; an eager call on a side stream allocates its
    own workspace there."""
    c = build(20, [3000, 1500], [1, 1], 8, 1, 128, 16, torch.bfloat16, window=1000)
    want = run(c, True, softcap=30.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(c, True, softcap=30.0, stream=side)
    assert torch.equal(got, want)
    ws = torch.empty(P.pa_decode_workspace_bytes(2, 8, 128, 3000, 16, 0), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pa_decode_mod(out, c.q, *c.pools, c.table, c.context_lens, c.scale, 1, 16, softcap=30.0,
                        window=1000, max_context_len=3000, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.context_lens[0] = 2100
    c.k_cache.nan_to_num_(0.0)              # tokens the shorter window now sees
    c.v_cache.nan_to_num_(0.0)
    c.table.clamp_(min=0)
    graph.replay()
    torch.cuda.synchronize()
    eager = run(c, True, softcap=30.0, max_context_len=3000)
    assert torch.equal(out, eager) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("dtype,fp8", [(torch.float16, False), (torch.bfloat16, True)])
def test_rows_without_a_sequence_stay_in_a_split_call(dtype, fp8):
    c = build(22, [500, 800], [10, 20], 4, 1, 128, 16, dtype, fp8)
    good = run(c, False, partition_size=128)
    c.query_start[2] = 25
    out = torch.full(c.q.shape, 7.0, dtype=torch.float32, device="cuda")
    f = P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod
    f(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, c.scale, 1, 16, max_query_len=20,
      max_context_len=800, partition_size=128)
    torch.cuda.synchronize()
    assert (out[25:] == 7.0).all() and torch.isfinite(out[:25]).all()
    assert torch.equal(out[:10], good[:10])
    assert P.pa_get_device_error() == 2


def test_bad_sequences_in_a_cut_last_wave():
    """As test_chunk_last_wave_is_cut, with lengths out of range among the units of one CTA and
    among the split ones: their rows become NaN, all others stay as they are."""
    lens = [1100 + 3 * i for i in range(17)] + [1300, 40, 1250, 1030]
    new = [40 - i % 3 for i in range(17)] + [40, 40, 0, 37]
    c = build(21, lens, new, 8, 8, 128, 16, torch.bfloat16)
    good = run(c, False, softcap=30.0)
    start = c.query_start.tolist()
    bad = [2, 18, 20]
    for s, L in zip(bad, (1301, -1, 36)):
        c.context_lens[s] = L
    out = run(c, False, softcap=30.0)
    assert P.pa_get_device_error() == 2
    for s in range(len(lens)):
        rows = slice(start[s], start[s + 1])
        assert torch.isnan(out[rows]).all() if s in bad else torch.equal(out[rows], good[rows])
