"""pa_append_fp8_block and pa_rotary_and_append_fp8_block against their definition.

V (and K that does not turn) is x / s with s a power of two: exact in fp32, so codes and scales are
equal bit for bit.  A turned K element is fp32 arithmetic on exact inputs: cos and sin within 2 ulp
(the phase is exact to 2^-33 turns), two products and a sum, so within 6 * 2^-24 (|a| + |b|) of the
exact value; its code may then be the other neighbour of a tie, and a scale the other power of two
where the largest magnitude lies that near its border.
"""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
TURN = 6 * 2.0 ** -24


def make(seed, lens, new, Hq, Hkv, D, B, dtype, spread=2.0):
    """Rows of one projection, pools full of stale codes (NaN among them) and scales."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    T = sum(new)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g) * torch.exp2(
        spread * torch.randn((T, Hq + 2 * Hkv, 1), generator=g))
    qkv = qkv.to(dtype)
    need = [(L + B - 1) // B for L in lens]
    N = sum(need) + 2
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    ids = rng.permutation(N)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    codes = [torch.tensor(rng.integers(0, 256, (N, Hkv, B, D)), dtype=torch.uint8) for _ in range(2)]
    stride = (Hkv + 3) // 4 * 4
    scales = [torch.exp2(torch.tensor(rng.integers(-9, -4, (N, stride)))).float() for _ in range(2)]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return qkv, codes, scales, table, start


def run(qkv, codes, scales, table, lens, start, Hq, Hkv, freq=None, q_out=None, positions=None, inter=False,
        mag=1.0, max_new=None):
    import paged_kv_cache_119_gb300 as pa
    x = qkv.cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    dev = [c.cuda() for c in codes] + [s.cuda() for s in scales]
    args = (k, v, *dev, torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            torch.tensor(start).cuda())
    out = None
    if freq is None:
        pa.pa_append_fp8_block(*args, max_query_len=max_new)
    else:
        out = torch.empty((x.shape[0], Hq, x.shape[2]), dtype=x.dtype, device="cuda") if q_out is None else q
        pos = None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda()
        pa.pa_rotary_and_append_fp8_block(out, q, *args, freq, positions=pos, interleaved=inter, magnitude=mag,
                                          max_query_len=max_new)
        out = out.cpu()
    torch.cuda.synchronize()
    return [t.cpu() for t in dev], out, x.cpu()


PATTERNS = {
    "step": ([17, 1, 16, 40, 33], [1, 1, 1, 1, 1]),
    "mixed": ([5, 100, 37, 64, 21, 3], [5, 1, 20, 64, 4, 0]),
    "one long": ([300, 7, 9, 1, 12, 60, 33, 2], [277, 1, 1, 1, 1, 1, 1, 1]),
}


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B,Hkv", [(128, 16, 8), (128, 32, 3), (64, 16, 5), (64, 32, 40)])
def test_append(pattern, dtype, D, B, Hkv):
    lens, new = PATTERNS[pattern]
    qkv, codes, scales, table, start = make(11, lens, new, 2, Hkv, D, B, dtype)
    want = [c.clone() for c in codes], [s.clone() for s in scales]
    for i, first in enumerate((2, 2 + Hkv)):
        R.append(qkv[:, first:first + Hkv], want[0][i], want[1][i], table, lens, new, B)
    got, _, _ = run(qkv, codes, scales, table, lens, start, 2, Hkv, max_new=max(new))
    for i in range(2):
        assert R.same(got[2 + i], want[1][i])
        assert R.same(got[i], want[0][i])


@pytest.mark.parametrize("pattern", PATTERNS)
def test_append_without_a_tight_bound(pattern):
    lens, new = PATTERNS[pattern]
    qkv, codes, scales, table, start = make(12, lens, new, 2, 4, 64, 16, torch.float16)
    tight, _, _ = run(qkv, codes, scales, table, lens, start, 2, 4, max_new=max(new))
    loose, _, _ = run(qkv, codes, scales, table, lens, start, 2, 4)
    assert all(R.same(a, b) for a, b in zip(tight, loose))


LAYOUTS = {"whole": (1.0, False), "pairs": (1.0, True), "half": (0.5, False), "half pairs": (0.5, True),
           "odd": (0.28125, False), "odd pairs": (0.28125, True)}


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,B,Hq,Hkv,dtype", [(128, 16, 8, 2, torch.bfloat16), (128, 32, 6, 3, torch.float16),
                                             (64, 16, 5, 5, torch.bfloat16), (64, 32, 12, 4, torch.float16)])
def test_rotary_append(pattern, layout, D, B, Hq, Hkv, dtype):
    lens, new = PATTERNS[pattern]
    share, inter = LAYOUTS[layout]
    rot = int(D * share) // 2 * 2
    mag = 1.25
    freq = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    qkv, codes, scales, table, start = make(13, lens, new, Hq, Hkv, D, B, dtype, spread=0.5)
    place = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
    far = place * 1009 + 100000
    for positions in (None, far):
        pos = torch.tensor(place if positions is None else far)
        got, q, _ = run(qkv, codes, scales, table, lens, start, Hq, Hkv, freq, positions=positions, inter=inter,
                        mag=mag, max_new=max(new))
        # q: fp32 arithmetic rounded once
        want = R.rotate(qkv[:, :Hq], pos, freq, inter, mag)
        reach = pair_size(qkv[:, :Hq], rot, inter) * mag
        err = (q.double() - want).abs()
        half = torch.finfo(dtype).eps / 2
        assert (err <= TURN * reach + half * (want.abs() + TURN * reach) + 2.0 ** -25).all()
        if rot < D:
            assert torch.equal(q[..., rot:], qkv[:, :Hq, rot:])
        # V bit for bit
        vc, vs = codes[1].clone(), scales[1].clone()
        R.append(qkv[:, Hq + Hkv:], vc, vs, table, lens, new, B)
        assert R.same(got[1], vc) and R.same(got[3], vs)
        # K: scales, then codes given the scales
        k = R.rotate(qkv[:, Hq:Hq + Hkv], pos, freq, inter, mag)
        check_turned(k, pair_size(qkv[:, Hq:Hq + Hkv], rot, inter) * mag, codes[0], scales[0], got[0], got[2],
                     table, lens, new, B)


def pair_size(x, rot, inter):
    """|a| + |b| of each element's pair (0 past the last pair)."""
    y = torch.zeros(x.shape, dtype=torch.float64)
    if rot:
        a = torch.arange(rot // 2) * (2 if inter else 1)
        b = a + (1 if inter else rot // 2)
        s = x.double()[..., a].abs() + x.double()[..., b].abs()
        y[..., a], y[..., b] = s, s
    return y


def check_turned(k, reach, codes, scales, got, got_scales, table, lens, new, B):
    """Scales and codes of turned rows, up to the rounding of the rotation; all else as it was."""
    untouched = torch.ones(codes.shape[0], dtype=torch.bool)
    value = R.decode(got)
    row = 0
    for s, (L, n) in enumerate(zip(lens, new)):
        at = L - n
        while at < L:
            lb = at // B
            end = min(L, lb * B + B)
            blk, r0, cnt = int(table[s, lb]), at - lb * B, end - at
            x, slack = k[row:row + cnt], TURN * reach[row:row + cnt]
            row += cnt
            at = end
            untouched[blk] = False
            for h in range(codes.shape[1]):
                top, sl = x[:, h].abs(), slack[:, h]
                ok = {max(R.scale_for(float(v)), float(scales[blk, h]) if r0 else 0.0)
                      for v in ((top - sl).max(), top.max(), (top + sl).max())}
                now = float(got_scales[blk, h])
                assert now in ok
                have = value[blk, h, r0:r0 + cnt]
                exact = x[:, h] / now
                step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp(min=2.0 ** -6))) - 3)
                inside = exact.abs() <= 448
                assert ((have - exact).abs() <= step / 2 * (1 + 2.0 ** -20) + sl / now)[inside].all()
                assert (have.abs() == 448)[~inside].all()
                if r0:
                    ratio = float(scales[blk, h]) / now
                    told = codes[blk, h, :r0] if ratio == 1 else R.encode(R.decode(codes[blk, h, :r0]) * ratio)
                    assert R.same(got[blk, h, :r0], told)
                assert R.same(got[blk, h, r0 + cnt:], codes[blk, h, r0 + cnt:])
    assert R.same(got[untouched], codes[untouched])
    assert R.same(got_scales[untouched], scales[untouched])


@pytest.mark.parametrize("layout", ["whole", "odd", "pairs"])
@pytest.mark.parametrize("new", [1, 9])
def test_q_in_place(layout, new):
    share, inter = LAYOUTS[layout]
    rot = int(128 * share) // 2 * 2
    freq = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    lens = [20, 50]
    qkv, codes, scales, table, start = make(14, lens, [new] * 2, 8, 2, 128, 16, torch.bfloat16)
    a, q, _ = run(qkv, codes, scales, table, lens, start, 8, 2, freq, inter=inter, max_new=new)
    b, q2, x = run(qkv, codes, scales, table, lens, start, 8, 2, freq, q_out="in place", inter=inter, max_new=new)
    assert torch.equal(q, q2) and torch.equal(x[:, :8], q2)
    assert torch.equal(x[:, 8:], qkv[:, 8:])
    assert all(R.same(u, w) for u, w in zip(a, b))


def test_values_at_the_ends():
    """Zeros, infinities, NaN, the largest and the smallest numbers, and a scale border."""
    lens, new, B, D, H = [16, 16, 16, 16, 16, 16], [16] * 6, 16, 128, 2
    qkv, codes, scales, table, start = make(15, lens, new, 2, H, D, B, torch.bfloat16)
    k = qkv[:, 2:2 + H]
    k[0:16] = 0                                              # nothing: the smallest scale
    k[16, 0, 3], k[17, 0, 5], k[18, 1, 7] = float("inf"), -float("inf"), float("nan")
    k[32:48] = torch.finfo(torch.bfloat16).max               # beyond 448 * 2^48
    k[48:64] = 2.0 ** -60                                    # below the smallest scale's codes
    k[64:80] = 0
    k[64, :, 0] = 448.0 * 2.0 ** -3                          # exactly on a border
    k[80:96] = 0
    k[80, :, 0] = 452.0 * 2.0 ** -3                          # the next number up (8 bits)
    want = codes[0].clone(), scales[0].clone()
    R.append(k, *want, table, lens, new, B)
    got, _, _ = run(qkv, codes, scales, table, lens, start, 2, H, max_new=16)
    assert R.same(got[2], want[1])
    assert R.same(got[0], want[0])
    block = [int(table[s, 0]) for s in range(6)]
    assert float(got[2][block[0], 0]) == 2.0 ** -48 and float(got[2][block[2], 0]) == 2.0 ** 48
    assert float(got[2][block[4], 0]) == 2.0 ** -3 and float(got[2][block[5], 0]) == 2.0 ** -2
    assert bool((got[0][block[1], 0, 0, 3] == 0x7e) and (got[0][block[1], 0, 1, 5] == 0xfe))
    assert int(got[0][block[1], 1, 2, 7]) & 0x7f == 0x7f


@pytest.mark.parametrize("old", [2.0 ** -7 * 1.37, 2.0 ** 60, 0.0, -1.0, float("nan"), float("inf")])
def test_earlier_scales_of_other_kinds(old):
    """A scale that no append wrote: any value counts as held within the bounds (NaN as the lower)."""
    lens, new, B = [20, 9], [3, 2], 16
    qkv, codes, scales, table, start = make(16, lens, new, 2, 3, 64, B, torch.float16)
    for s in scales:
        s.fill_(old)
    held = 2.0 ** -48 if old != old else min(max(old, 2.0 ** -48), 2.0 ** 48)
    want = [c.clone() for c in codes], [torch.where(torch.ones_like(s) > 0, held, s) for s in scales]
    for i, first in enumerate((2, 5)):
        R.append(qkv[:, first:first + 3], want[0][i], want[1][i], table, lens, new, B)
    got, _, _ = run(qkv, codes, scales, table, lens, start, 2, 3, max_new=3)
    for i in range(2):
        for s in range(2):
            blk = int(table[s, (lens[s] - 1) // B])
            assert R.same(got[2 + i][blk, :3], want[1][i][blk, :3])
            assert R.same(got[i][blk], want[0][i][blk])


def test_one_by_one_and_all_at_once():
    """Scales agree, and codes but for those that fell below 2^-6 on the way."""
    B, D, H, L = 16, 64, 4, 45
    qkv, codes, scales, table, start = make(17, [L], [L], 2, H, D, B, torch.bfloat16, spread=1.5)
    once, _, _ = run(qkv, codes, scales, table, [L], start, 2, H, max_new=L)
    at = [c.clone() for c in codes] + [s.clone() for s in scales]
    for t in range(L):
        at, _, _ = run(qkv[t:t + 1], at[:2], at[2:], table, [t + 1], np.array([0, 1], np.int32), 2, H, max_new=1)
    for i in range(2):
        assert torch.equal(at[2 + i], once[2 + i])
        a, b = R.decode(at[i]), R.decode(once[i])
        used = torch.zeros(a.shape, dtype=torch.bool)
        for t in range(L):
            used[int(table[0, t // B]), :, t % B] = True
        big = used & (b.abs() > 2.0 ** -6)
        assert torch.equal(a[big], b[big]) and big.sum() > 1000
        # two roundings to multiples of 2^-9 at most on the way down, each half a step
        assert ((a - b).abs()[used & ~big] <= 2.0 ** -9).all()


def test_bad_blocks_lengths_and_rows():
    import paged_kv_cache_119_gb300 as pa
    from paged_kv_cache_119_gb300 import _native as N
    lens, new, B, H = [20, 40, 10], [4, 8, 2], 16, 2
    qkv, codes, scales, table, start = make(18, lens, new, 2, H, 64, B, torch.float16)
    freq = [1.0, 0.5]
    good, q, _ = run(qkv, codes, scales, table, lens, start, 2, H, freq, max_new=8)
    assert pa.pa_get_device_error() == 0

    def changed(**kw):
        a = dict(table=table, lens=lens, start=start, max_new=8)
        a.update(kw)
        return run(qkv, codes, scales, a["table"], a["lens"], a["start"], 2, H, freq, max_new=a["max_new"])

    for bad_id in (-1, codes[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 2] = bad_id                      # tokens 32 .. 39, all of sequence 1's
        got, q2, _ = changed(table=t)
        assert pa.pa_get_device_error() == N.PA_DEVERR_BLOCK_ID
        assert torch.equal(q, q2)
        blk = int(table[1, 2])
        for i in range(4):
            want = good[i].clone()
            want[blk] = (codes + scales)[i][blk]
            assert R.same(got[i], want)
    for kw in (dict(lens=[20, 7, 10]), dict(lens=[20, -3, 10]), dict(lens=[20, 10 ** 9, 10]), dict(max_new=7)):
        got, _, _ = changed(**kw)
        assert pa.pa_get_device_error() == N.PA_DEVERR_CONTEXT_LEN
        touched = [int(table[0, 1]), int(table[2, 0])]          # the two sound sequences' blocks
        rest = torch.ones(codes[0].shape[0], dtype=torch.bool)
        rest[touched] = False
        for i in range(4):
            assert R.same(got[i][touched], good[i][touched])
            assert R.same(got[i][rest], (codes + scales)[i][rest])
    # rows behind the last sequence: flagged and left alone
    got, _, _ = changed(start=np.array([0, 4, 12, 13], np.int32), lens=[20, 40, 9])
    assert pa.pa_get_device_error() == N.PA_DEVERR_CONTEXT_LEN
    # a malformed query_start reaches nothing out of range
    for st in ([0, -5, 12, 14], [0, 4, 2, 14], [0, 4, 99, 14], [9, 4, 2, 1], [-8, 4, 12, 14]):
        changed(start=np.array(st, np.int32))
        assert pa.pa_get_device_error() & N.PA_DEVERR_CONTEXT_LEN


def test_python_refusals():
    import paged_kv_cache_119_gb300 as pa
    lens, new = [20, 40], [4, 8]
    qkv, codes, scales, table, start = make(19, lens, new, 2, 2, 64, 16, torch.float16)
    x = qkv.cuda()
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    base = dict(k=k, v=v, k_cache=codes[0].cuda(), v_cache=codes[1].cuda(), k_scales=scales[0].cuda(),
                v_scales=scales[1].cuda(), block_tables=torch.tensor(table).cuda(),
                context_lens=torch.tensor(lens, dtype=torch.int32).cuda(), query_start=torch.tensor(start).cuda())
    for kw, err in [(dict(k_scales=scales[0]), ValueError), (dict(k_scales=scales[0].cuda()[:, :1]), ValueError),
                    (dict(k_scales=scales[0].cuda().double()), ValueError),
                    (dict(v_scales=scales[0].cuda()[:-1]), ValueError),
                    (dict(k_cache=codes[0].cuda().float()), TypeError), (dict(v=v[:, :1]), ValueError),
                    (dict(k=k.transpose(1, 2)), ValueError), (dict(context_lens=torch.tensor(lens).cuda()), TypeError),
                    (dict(query_start=torch.tensor(start[:-1]).cuda()), ValueError),
                    (dict(k=k.float(), v=v.float()), Exception)]:
        with pytest.raises(err):
            pa.pa_append_fp8_block(**{**base, **kw})
    out = torch.empty((12, 2, 64), dtype=torch.float16, device="cuda")
    for kw, err in [(dict(q_out=out.bfloat16()), TypeError), (dict(q=q[:5]), ValueError),
                    (dict(positions=torch.zeros(5, dtype=torch.int32, device="cuda")), ValueError),
                    (dict(positions=torch.zeros(12, device="cuda")), TypeError), (dict(inv_freq=[]), Exception)]:
        with pytest.raises(err):
            pa.pa_rotary_and_append_fp8_block(**{**dict(q_out=out, q=q, inv_freq=[1.0]), **base, **kw})
