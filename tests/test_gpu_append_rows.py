"""Appends with rows that no sequence owns, with many sequences, and with a malformed query_start: what
is flagged, what is written and what stays as it was.  Codes and scales are compared bit for bit with
the definition; a padding row of q_out keeps what it held."""
import numpy as np
import pytest
import torch

import block_reference as R
from test_gpu_append import make

pytestmark = pytest.mark.gpu

B, D, HQ, HKV = 16, 64, 3, 2
# direct: every sequence gets as many units; searched: one long prompt among short ones
SHAPES = {"step": ([17, 1, 16, 40, 33], [1] * 5), "direct": ([20, 40, 10], [4, 8, 2]),
          "searched": ([300, 7, 9, 1, 12, 60, 33, 2], [277, 1, 1, 1, 1, 1, 1, 1])}
FREQ = [1.0, 0.25]


def append(qkv, codes, scales, table, lens, start, turn, max_new):
    """The pools after the call, and q_out, which held 7 everywhere."""
    import paged_kv_cache_119_gb300 as pa
    x = qkv.cuda()
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    pools = [t.cuda() for t in codes] + [t.cuda() for t in scales]
    args = (k, v, *pools, torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            torch.tensor(np.asarray(start, np.int32)).cuda())
    out = torch.full((x.shape[0], HQ, D), 7.0, dtype=x.dtype, device="cuda")
    if turn:
        pa.pa_rotary_and_append_fp8_block(out, q, *args, FREQ, max_query_len=max_new)
    else:
        pa.pa_append_fp8_block(*args, max_query_len=max_new)
    torch.cuda.synchronize()
    return [t.cpu() for t in pools], out.cpu(), pa.pa_get_device_error()


def expect(qkv, codes, scales, table, lens, new):
    want = [c.clone() for c in codes] + [s.clone() for s in scales]
    for i, first in enumerate((HQ, HQ + HKV)):
        R.append(qkv[:, first:first + HKV], want[i], want[2 + i], table, lens, new, B)
    return want


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("before,behind", [(2, 0), (0, 3), (2, 3), (0, 0)])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_of_no_sequence(shape, before, behind, turn):
    from paged_kv_cache_119_gb300 import _native as N
    lens, new = SHAPES[shape]
    qkv, codes, scales, table, start = make(71, lens, new, HQ, HKV, D, B, torch.float16)
    pad = torch.full((before + behind, *qkv.shape[1:]), 100.0, dtype=qkv.dtype)
    rows = torch.cat([pad[:before], qkv, pad[before:]])
    got, out, flags = append(rows, codes, scales, table, lens, start + before, turn, max(new))
    assert flags == (N.PA_DEVERR_CONTEXT_LEN if before + behind else 0)
    want = expect(qkv, codes, scales, table, lens, new)
    for i in (1, 3) if turn else range(4):        # (turned K: test_gpu_append.py)
        assert R.same(got[i], want[i])
    own = out[before:before + qkv.shape[0]]
    assert (out[:before] == 7).all() and (out[before + qkv.shape[0]:] == 7).all()
    if turn:
        alone, q_alone, flags = append(qkv, codes, scales, table, lens, start, turn, max(new))
        assert flags == 0 and torch.equal(own, q_alone)
        assert all(R.same(a, b) for a, b in zip(got, alone))


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("start", [[5, 8, 9, 10], [100, 110, 112, 114], [-100, 4, 12, 14], [0, -300, 12, 14],
                                   [0, 4, 2 ** 31 - 1, 14], [-2 ** 31, 2 ** 31 - 1, 12, 14], [14, 14, 14, 14],
                                   [2 ** 31 - 1] * 4, [-2 ** 31] * 4])
@pytest.mark.parametrize("max_new", [8, 1000])
def test_a_malformed_start_is_flagged(start, max_new, turn):
    """Whether units are searched for (a loose bound) or not; blocks of no sequence stay as they were."""
    from paged_kv_cache_119_gb300 import _native as N
    lens, new = [20, 40, 10], [4, 8, 2]
    qkv, codes, scales, table, _ = make(72, lens, new, HQ, HKV, D, B, torch.float16)
    got, out, flags = append(qkv, codes, scales, table, lens, start, turn, max_new)
    assert flags == N.PA_DEVERR_CONTEXT_LEN
    used = torch.zeros(codes[0].shape[0], dtype=torch.bool)
    for s, L in enumerate(lens):
        used[torch.tensor(table[s, :(L + B - 1) // B]).long()] = True
    for i in range(4):
        assert R.same(got[i][~used], (codes + scales)[i][~used])


def many(where, count=300, long=600):
    """One long prompt among sequences of no or few tokens."""
    rng = np.random.default_rng(73)
    new = [int(n) for n in rng.choice([0, 1, 1, 1, 2], count)]
    new[{"first": 0, "middle": count // 2, "last": count - 1}[where]] = long
    lens = [n + int(e) for n, e in zip(new, rng.integers(0, 40, count))]
    return lens, new


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("count", [33, 300, 1200])
def test_many_sequences_beside_a_long_one(where, count):
    """The search of the units narrows 33 ways at a time."""
    lens, new = many(where, count)
    qkv, codes, scales, table, start = make(74, lens, new, HQ, HKV, D, B, torch.bfloat16)
    want = expect(qkv, codes, scales, table, lens, new)
    got, _, flags = append(qkv, codes, scales, table, lens, start, False, max(new))
    assert flags == 0
    for i in range(4):
        assert R.same(got[i], want[i])


@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_many_turned_sequences_beside_a_long_one(where):
    """As the same sequences one at a time."""
    lens, new = many(where)
    qkv, codes, scales, table, start = make(75, lens, new, HQ, HKV, D, B, torch.bfloat16)
    got, q, flags = append(qkv, codes, scales, table, lens, start, True, max(new))
    assert flags == 0
    at = [c.clone() for c in codes] + [s.clone() for s in scales]
    for s in list(range(0, len(lens), 11)) + [0, len(lens) // 2, len(lens) - 1]:
        n = new[s]
        if n == 0:
            continue
        rows = slice(int(start[s]), int(start[s]) + n)
        one, q1, flags = append(qkv[rows], at[:2], at[2:], table[s:s + 1], lens[s:s + 1], [0, n], True, n)
        assert flags == 0 and torch.equal(q[rows], q1)
        blocks = torch.tensor(table[s, (lens[s] - n) // B:(lens[s] + B - 1) // B]).long()
        for i in range(4):
            assert R.same(got[i][blocks], one[i][blocks])


def test_lengths_out_of_range_among_many():
    """Skipped and flagged; all others as they would be without them."""
    from paged_kv_cache_119_gb300 import _native as N
    lens, new = many("middle")
    qkv, codes, scales, table, start = make(76, lens, new, HQ, HKV, D, B, torch.float16)
    good = expect(qkv, codes, scales, table, lens, new)
    taken = [s for s in range(len(lens)) if new[s] > 0]
    for s, L in ((taken[0], -1), (taken[7], 10 ** 9), (150, 599), (taken[-1], 0)):
        bad = list(lens)
        bad[s] = L
        got, _, flags = append(qkv, codes, scales, table, bad, start, False, max(new))
        assert flags == N.PA_DEVERR_CONTEXT_LEN
        blocks = torch.tensor(table[s, (lens[s] - new[s]) // B:(lens[s] + B - 1) // B]).long()
        for i in range(4):
            want = good[i].clone()
            want[blocks] = (codes + scales)[i][blocks]
            assert R.same(got[i], want)
