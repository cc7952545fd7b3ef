"""A row whose every block is invalid is NaN also where its parts are merged (split calls and
the shared-prefix decode), as it is in an unsplit call: the parts of such a row hold no token
at all, and must not pass for a row that sees nothing."""
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


# one of each kernel: CUDA cores, mma.sync with 4 and 8 rows, the row kernel, tcgen05 on codes
SHAPES = [(2, 2, 128, torch.float16, False), (8, 2, 64, torch.bfloat16, False),
          (8, 1, 128, torch.float16, False), (16, 1, 128, torch.bfloat16, False),
          (2, 2, 128, torch.bfloat16, True), (8, 2, 128, torch.float16, True),
          (8, 1, 128, torch.bfloat16, True), (16, 1, 128, torch.float16, True),
          (2, 2, 64, torch.float16, True), (8, 1, 64, torch.bfloat16, True)]


def expect(out, rows, c, ref=None):
    """NaN in `rows` and nowhere else, the invalid blocks flagged; the other rows against ref."""
    assert P.pa_get_device_error() == 1
    ok = [r for r in range(out.shape[0]) if r not in rows]
    assert torch.isnan(out[sorted(rows)]).all()
    want, vmax = reference(c) if ref is None else ref
    check(out[ok], want[ok], vmax, CHUNK_TOL)


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", SHAPES + [(2, 2, 64, torch.float32, False)])
def test_split_decode(Hq, Hkv, D, dtype, fp8, bad):
    c = build(1, [300, 290, 9, 400], [1] * 4, Hq, Hkv, D, 16, dtype, fp8)
    c.table[1] = bad
    c.table[2] = bad
    f = P.pa_decode_mod_fp8 if fp8 else P.pa_decode_mod
    for part in (128, -1):
        out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
        f(out, c.q, *c.pools, c.table, c.context_lens, c.scale, c.Hkv, c.B, partition_size=part)
        expect(out, {1, 2}, c)


@pytest.mark.parametrize("new", [[3, 5, 2], [40, 50, 9]], ids=["few", "long"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", SHAPES)
def test_split_chunk(Hq, Hkv, D, dtype, fp8, new):
    c = build(2, [300, 290, 260], new, Hq, Hkv, D, 16, dtype, fp8)
    c.table[1] = -1
    f = P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod
    rows = set(range(new[0], new[0] + new[1]))
    for part in (128, -1):
        out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
        f(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, c.scale, c.Hkv, c.B,
          max_query_len=max(new), partition_size=part)
        expect(out, rows, c)


def prefix_case(groups, Hq, Hkv, D, B, dtype, fp8, seed=3):
    """groups: list of (shared tokens, [own tokens])."""
    lens, shared, start = [], [], [0]
    for prefix, tails in groups:
        shared.append((len(lens), len(lens) + len(tails), prefix))
        lens += [prefix + t for t in tails]
        start.append(len(lens))
    c = build(seed, lens, [1] * len(lens), Hq, Hkv, D, B, dtype, fp8, shared=shared)
    c.prefix_lens = torch.tensor(c.shared_len, device="cuda")
    c.group_start = torch.tensor(start, dtype=torch.int32, device="cuda")
    c.bounds = dict(max_group_size=max(len(t) for _, t in groups),
                    max_prefix_len=max(p for p, _ in groups),
                    max_suffix_len=max(max(t) for _, t in groups))
    return c


def prefix_run(c, **kw):
    out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    f = P.pa_decode_prefix_fp8 if c.fp8 else P.pa_decode_prefix
    f(out, c.q, *c.pools, c.table, c.context_lens, c.prefix_lens, c.group_start, c.scale, c.Hkv, c.B,
      **{**c.bounds, **kw})
    return out


@pytest.mark.parametrize("members", [3, 40], ids=["rows", "wide"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", SHAPES)
def test_prefix_decode(Hq, Hkv, D, dtype, fp8, members):
    """Sequence 0 shares nothing; the first group's members own nothing (one of them) or some
    tokens; the last group is sound."""
    groups = [(0, [40]), (64, [0] + [7] * (members - 1)), (64, [5, 300])]
    for part in (0, -1, 128):
        c = prefix_case(groups, Hq, Hkv, D, 16, dtype, fp8)
        ref = reference(c)
        c.table[0] = -1                              # no block of its own
        expect(prefix_run(c, partition_size=part), {0}, c, ref)
        c = prefix_case(groups, Hq, Hkv, D, 16, dtype, fp8)
        c.table[1, :4] = 10 ** 6                     # no block of the shared prefix
        expect(prefix_run(c, partition_size=part), set(range(1, 1 + members)), c, ref)
        c = prefix_case(groups, Hq, Hkv, D, 16, dtype, fp8)
        c.table[members + 2, 4:] = -1                # a valid prefix, no own block
        expect(prefix_run(c, partition_size=part), {members + 2}, c, ref)


@pytest.mark.parametrize("tails", [[9] * 30, [9]], ids=["wide", "single"])
def test_a_prefix_of_no_whole_blocks(tails):
    """The whole group agrees on a length that ends inside a block."""
    c = prefix_case([(64, [3, 4]), (96, tails), (32, [1])], 8, 2, 128, 16, torch.bfloat16, False)
    ref, vmax = reference(c)
    bad = range(2, 2 + len(tails))
    c.prefix_lens[2:2 + len(tails)] -= 8
    out = prefix_run(c)
    assert P.pa_get_device_error() & 2
    ok = [s for s in range(len(c.lens)) if s not in bad]
    assert torch.isnan(out[list(bad)]).all()
    check(out[ok], ref[ok], vmax, CHUNK_TOL)
