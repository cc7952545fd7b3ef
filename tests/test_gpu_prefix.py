"""Shared-prefix decode (pa_decode_prefix and its E4M3 form) on the GPU against a plain
64-bit reference: tolerances are derived in attn_reference.py (the prefix of a large group
runs on the tcgen05 chunk kernel: CHUNK_TOL)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import CHUNK_TOL, build, check, reference

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


def make(seed, groups, Hq, Hkv, D, B, dtype, fp8=False, kstd=1.0):
    """groups: list of (shared tokens, [suffix lengths])."""
    lens, shared, start = [], [], [0]
    for prefix, tails in groups:
        a = len(lens)
        lens += [prefix + t for t in tails]
        shared.append((a, len(lens), prefix))
        start.append(len(lens))
    c = build(seed, lens, [1] * len(lens), Hq, Hkv, D, B, dtype, fp8, shared=shared, kstd=kstd)
    c.prefix_lens = torch.tensor(c.shared_len, device="cuda")
    c.group_start = torch.tensor(start, dtype=torch.int32, device="cuda")
    c.bounds = dict(max_group_size=max(len(t) for _, t in groups),
                    max_prefix_len=max(p for p, _ in groups),
                    max_suffix_len=max(max(t) for _, t in groups))
    return c


def run(c, out_dtype=torch.float32, partition_size=0, stream=None, workspace=None, **bounds):
    out = torch.full(c.q.shape, float("nan"), dtype=out_dtype, device="cuda")
    f = P.pa_decode_prefix_fp8 if c.fp8 else P.pa_decode_prefix
    f(out, c.q, *c.pools, c.table, c.context_lens, c.prefix_lens, c.group_start, c.scale, c.Hkv, c.B,
      partition_size=partition_size, stream=stream, workspace=workspace, **{**c.bounds, **bounds})
    torch.cuda.synchronize()
    return out


def compare(c, **kw):
    out = run(c, **kw)
    assert P.pa_get_device_error() == 0
    check(out, *reference(c), CHUNK_TOL)
    return out


SMALL = [(64, [1, 5, 70]), (0, [40]), (160, [0, 33]), (32, [9])]
MEDIUM = [(320, [5, 0, 90, 33, 17, 1, 64]), (48, [2, 2, 2]), (0, [100])]     # up to 32 rows at G = 4
WIDE = [(192, [int(x) for x in np.random.default_rng(1).integers(0, 90, 37)]), (96, [20, 1])]
SHAPES = [(4, 4, 128, 16, torch.float16, False), (8, 2, 64, 32, torch.bfloat16, False),
          (8, 1, 128, 16, torch.bfloat16, False), (14, 2, 128, 32, torch.float16, False),
          (6, 2, 64, 16, torch.float16, False), (4, 2, 128, 16, torch.bfloat16, False),
          (2, 2, 128, 16, torch.bfloat16, True), (8, 2, 128, 32, torch.float16, True),
          (8, 1, 128, 16, torch.bfloat16, True), (3, 1, 128, 32, torch.bfloat16, True),
          (2, 2, 64, 16, torch.float16, True), (8, 1, 64, 32, torch.bfloat16, True)]


@pytest.mark.parametrize("groups", [SMALL, MEDIUM, WIDE], ids=["small", "medium", "wide"])
@pytest.mark.parametrize("Hq,Hkv,D,B,dtype,fp8", SHAPES)
def test_against_the_reference(Hq, Hkv, D, B, dtype, fp8, groups):
    groups = [(p // B * B, tails) for p, tails in groups]
    c = make(Hq + D, groups, Hq, Hkv, D, B, dtype, fp8)
    for part in (0, -1, 128):
        compare(c, partition_size=part)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_native_output(dtype):
    c = make(2, WIDE, 8, 2, 128, 16, dtype)
    compare(c, out_dtype=dtype)


@pytest.mark.parametrize("Hq,fp8", [(8, False), (4, False), (8, True), (2, True)])
def test_long_prefix_automatic_split(Hq, fp8):
    c = make(3, [(6016, [1, 700, 300] * 4), (2048, [1300])], Hq, 1, 128, 32, torch.bfloat16, fp8)
    compare(c)


def test_more_rows_than_one_tile():
    """A group whose (sequence, head) rows fill several 256-row CTAs."""
    c = make(4, [(320, [3] * 70)], 16, 2, 128, 16, torch.bfloat16)
    compare(c)


def test_every_token_counts_once():
    """Equal scores: the mean of V over prefix and suffix, n 2^-23 max |v| for the sums."""
    for fp8 in (False, True):
        for groups in (SMALL, WIDE):
            c = make(5, groups, 8, 2, 128, 16, torch.float16, fp8, kstd=0.0)
            ref, vmax = reference(c)
            for part in (0, 128):
                err = np.abs(run(c, partition_size=part).double().cpu().numpy() - ref).max()
                assert err <= 300 * 2.0 ** -23 * vmax, err


def test_agrees_with_the_plain_decode():
    c = make(6, [(512, [30, 40, 50, 1])] * 3, 8, 2, 128, 16, torch.float16)
    a = run(c)
    b = torch.empty_like(a)
    P.pa_decode(b, c.q, *c.pools, c.table, c.context_lens, c.scale, c.Hkv, c.B)
    vmax = max(v.abs().max().item() for v in c.V)
    assert (a - b).abs().max() <= 2.0 ** -11 * vmax + 1e-4


def test_nothing_shared_and_nothing_own():
    c = make(7, [(0, [5, 17, 0])], 4, 2, 64, 16, torch.bfloat16)       # an empty context: zeros
    out = compare(c)
    assert (out[2] == 0).all()
    c = make(8, [(64, [0, 0])], 4, 2, 64, 16, torch.bfloat16)          # prefix only
    compare(c, max_suffix_len=0)


def bad_rows(c, which, **kw):
    out = run(c, **kw)
    assert P.pa_get_device_error() & 2
    ok = [s for s in range(len(c.lens)) if s not in which]
    assert torch.isnan(out[list(which)]).all()
    ref, vmax = reference(c)
    check(out[ok], ref[ok], vmax, CHUNK_TOL)


@pytest.mark.parametrize("groups", [SMALL, [(64, [9] * 30), (32, [1, 2])]], ids=["small", "wide"])
def test_bad_lengths_and_groups(groups):
    n0 = len(groups[0][1])
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    last = len(c.lens) - 1
    c.prefix_lens[n0 - 1] += 16                     # a member that disagrees
    bad_rows(c, {n0 - 1})
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    c.context_lens[0] = 63                          # shorter than its prefix
    bad_rows(c, {0})
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    bad_rows(c, {s for s in range(len(c.lens)) if c.shared_len[s] > 32}, max_prefix_len=32)
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    c.group_start[-1] -= 1                          # the last sequence belongs to no group
    bad_rows(c, {last})
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    big = max(len(t) for _, t in groups)
    bad = {s for s in range(len(c.lens)) for a, b in zip(c.group_start.tolist(), c.group_start.tolist()[1:])
           if a <= s < b and b - a == big}
    bad_rows(c, bad, max_group_size=big - 1)
    c = make(9, groups, 8, 2, 128, 16, torch.bfloat16)
    c.prefix_lens[last] = c.prefix_lens[last] - 8   # no whole number of blocks
    if len(groups[-1][1]) == 1:
        bad_rows(c, {last})


def test_bad_block_ids():
    c = make(10, SMALL, 8, 2, 128, 16, torch.float16)
    c.table[0, 1] = -5                              # shared by the first group
    out = run(c)
    assert P.pa_get_device_error() == 1
    assert torch.isnan(out[:3]).all() and torch.isfinite(out[3:]).all()
    c = make(10, SMALL, 8, 2, 128, 16, torch.float16)
    c.table[2, 64 // 16] = 10 ** 6                  # the third sequence's own
    out = run(c)
    assert P.pa_get_device_error() == 1
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all() and torch.isfinite(out[3:]).all()


def test_refusals():
    c = make(11, SMALL, 4, 2, 128, 16, torch.float16)
    for kw in (dict(max_prefix_len=100), dict(max_group_size=0), dict(max_group_size=99),
               dict(max_suffix_len=-1), dict(partition_size=64), dict(max_prefix_len=1 << 20),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(RuntimeError):
            run(c, **kw)
    c.prefix_lens = c.prefix_lens.long()
    with pytest.raises(TypeError):
        run(c)
    f32 = make(11, SMALL, 4, 2, 128, 16, torch.float32)
    with pytest.raises(RuntimeError):
        run(f32)


def test_captured_and_replayed_with_other_lengths():
    c = make(12, [(1024, [40, 100, 3, 77])] * 2, 8, 2, 128, 16, torch.bfloat16)
    want = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(run(c, stream=side), want)
    ws = torch.empty(P.pa_decode_prefix_workspace_bytes(8, 8, 128, 1024, 100), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pa_decode_prefix(out, c.q, *c.pools, c.table, c.context_lens, c.prefix_lens, c.group_start, c.scale,
                           c.Hkv, c.B, workspace=ws, **c.bounds)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.context_lens[1] = 1024 + 9
    c.prefix_lens[:4] = 512                         # the first group now shares less
    c.context_lens[0] = 512 + 30
    c.context_lens[1] = 512 + 90
    c.context_lens[2] = 512 + 1
    c.context_lens[3] = 512 + 64
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run(c))
    assert torch.equal(out[4:], want[4:])
