"""pa_rotary_and_cache and its E4M3 form on the GPU against the formula in 64 bits.

The reference reduces each angle exactly (rational arithmetic) before its cosine, so far
positions are checked at full accuracy.

Tolerance, derived: the kernel's half-turn argument is one fp32 rounding (|x| <= 1: at most
2^-25, i.e. pi 2^-25 = 9.4e-8 rad), sincospif is within 2 units of 2^-24 of values up to 1
(1.2e-7), the product with the magnitude rounds once (6e-8): 2.8e-7 on each of cos and sin,
and a product and a fused multiply-add round twice more (6e-8 each), so a result is within
4e-7 m (|x_a| + |x_b|) of the formula before its one rounding to the row type: half a step,
eps / 2 relative (absolute 2^-25 below f16's normal range).
"""
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_119_gb300 as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

getcontext().prec = 60
INV_2PI = Fraction(Decimal("0.15915494309189533576888376337251436203445964574046"))


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_119_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def clear_error_word(built):
    P.pa_get_device_error()
    yield


def cos_sin(positions, freq):
    """[T, R/2] in 64 bits: the fraction of a turn is exact before it is rounded."""
    step = [Fraction(float(f)) * INV_2PI for f in freq]
    turns = np.array([[float((int(n) * s) % 1) for s in step] for n in positions])
    return np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)


def rotate(x, cos, sin, inter, magnitude):
    """(turned rows, tolerance before the last rounding) in 64 bits; x [T, H, D]."""
    x = x.double().cpu().numpy()
    half = cos.shape[1]
    a = np.arange(half) * (2 if inter else 1)
    b = a + (1 if inter else half)
    y, tol = x.copy(), np.zeros_like(x)
    c, s = cos[:, None] * magnitude, sin[:, None] * magnitude
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    t = 4e-7 * abs(magnitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a] = t
    tol[..., b] = t
    return y, tol


def assert_rounded(got, ref, tol):
    """got is ref, within tol, rounded once to got's type."""
    eps = torch.finfo(got.dtype).eps / 2
    floor = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol + eps * (np.abs(ref) + tol) + floor).all(), float((err - tol).max())


def make(T, Hq, Hkv, D, B, dtype, seed, fused=True, pos_max=4096, slack=1.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if fused:
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dtype)
        q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    else:
        q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    N = int(np.ceil(T * slack / B)) + 1
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    slots[::7] = -1 - rng.integers(0, 5, len(slots[::7]))
    positions = rng.integers(0, pos_max, T)
    return q, k, v, N, slots, positions


def run(case, dtype=torch.bfloat16, T=19, Hq=8, Hkv=2, D=128, B=16, rot=128, inter=False, magnitude=1.0,
        fp8=False, fused=True, positions=None, inplace=False, freq=None, seed=1):
    q, k, v, N, slots, pos = make(T, Hq, Hkv, D, B, dtype, seed, fused)
    pos = pos if positions is None else np.asarray(positions)
    freq = P.pa_rotary_frequencies(rot) if freq is None else freq
    cos, sin = cos_sin(pos, freq)
    ref_q, tol_q = rotate(q, cos, sin, inter, magnitude)
    ref_k, tol_k = rotate(k, cos, sin, inter, magnitude)
    vh, kbits = v.clone(), k.clone()
    fill = torch.randint(0, 120, (N, Hkv, B, D), device="cuda", dtype=torch.uint8)
    kc = fill.view(torch.float8_e4m3fn).clone() if fp8 else fill.to(dtype)
    vc = kc.clone()
    before = kc.clone()
    qo = q if inplace else torch.empty((T, Hq, D), device="cuda", dtype=dtype)
    st, pt = torch.tensor(slots, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda")
    if fp8:
        ks = torch.rand(Hkv, device="cuda") * 0.02 + 0.005
        vs = torch.rand(Hkv, device="cuda") * 0.02 + 0.005
        P.pa_rotary_and_cache_fp8(qo, q, k, v, kc, vc, st, pt, freq, ks, vs, interleaved=inter,
                                  magnitude=magnitude)
    else:
        P.pa_rotary_and_cache(qo, q, k, v, kc, vc, st, pt, freq, interleaved=inter, magnitude=magnitude)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    assert_rounded(qo, ref_q, tol_q)
    assert torch.equal(k, kbits) and torch.equal(v, vh)          # the inputs stay
    live = np.flatnonzero(slots >= 0)
    blk, off = slots[live] // B, slots[live] % B
    untouched = np.ones((N, B), bool)
    untouched[blk, off] = False
    as_bytes = (lambda c: c.view(torch.uint8 if fp8 else torch.int32 if dtype == torch.float32 else torch.int16)
                .transpose(1, 2).cpu().numpy())
    for c in (kc, vc):                                           # every other slot keeps its bytes
        assert np.array_equal(as_bytes(c)[untouched], as_bytes(before)[untouched])
    rows = kc.transpose(1, 2)[blk, off] if not fp8 else \
        kc.view(torch.uint8).transpose(1, 2)[blk, off].view(torch.float8_e4m3fn)
    vrows = vc.view(torch.uint8).transpose(1, 2)[blk, off].view(torch.float8_e4m3fn) if fp8 else \
        vc.transpose(1, 2)[blk, off]
    if not fp8:
        assert_rounded(rows, ref_k[live], tol_k[live])
        assert torch.equal(vrows, vh[live])
        return
    # codes: monotone rounding, so between the codes of value -+ tolerance (fp32 division
    # adds one rounding, 2^-24 relative)
    for got, ref, tol, scale in ((rows, ref_k[live], tol_k[live], ks),
                                 (vrows, vh[live].double().cpu().numpy(), 0.0, vs)):
        x = ref / scale.double().cpu().numpy()[:, None]
        t = tol / scale.double().cpu().numpy()[:, None] + 2.0 ** -23 * np.abs(x)
        lo, hi = (torch.from_numpy(np.clip(x + d, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
                  for d in (-t, t))
        c = got.double().cpu().numpy()
        assert ((c >= lo) & (c <= hi)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_types(dtype, inter, fp8):
    run("types", dtype=dtype, inter=inter, fp8=fp8)


@pytest.mark.parametrize("D,rot", [(128, 64), (128, 36), (64, 64), (64, 2), (64, 20), (96, 96), (256, 256),
                                   (80, 32), (112, 24)])
@pytest.mark.parametrize("inter", [False, True])
def test_part_of_the_head(D, rot, inter):
    """Whole vectors, pairs that do not line up with 16-byte vectors, the smallest part."""
    run("part", D=D, rot=rot, inter=inter)
    run("part", D=D, rot=rot, inter=inter, fp8=True, dtype=torch.float16)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 64, 8), (2, 40, 40), (700, 5, 1), (97, 28, 4)])
def test_sizes(T, Hq, Hkv):
    run("sizes", T=T, Hq=Hq, Hkv=Hkv)


@pytest.mark.parametrize("B", [1, 16, 32, 48])
def test_block_sizes_and_dense_rows(B):
    run("dense", B=B, fused=False)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 36])
def test_far_and_negative_positions(inter, rot):
    """Angles of up to 2^31 radians: the fraction of a turn is exact."""
    pos = [0, 1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -5, 131071, 1048575, 65536, 3]
    run("far", T=len(pos), positions=pos, inter=inter, rot=rot, dtype=torch.float32)


def test_magnitude_and_scaled_frequencies():
    for scaling in ("linear", "ntk", "by_parts"):
        f = P.pa_rotary_frequencies(128, base=500000.0, scaling=scaling, factor=8.0, original_len=8192)
        run("scaled", freq=f, magnitude=1.2079, positions=np.arange(19) * 6899)
    run("flipped", magnitude=-0.5, freq=-P.pa_rotary_frequencies(128) * 37.0)   # any finite angle


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 64, 36])
@pytest.mark.parametrize("fused", [False, True])
def test_in_place(inter, rot, fused):
    run("inplace", inplace=True, inter=inter, rot=rot, fused=fused)


def test_values_that_are_not_finite_stay_in_their_pair():
    """An infinity or NaN in one pair of one head leaves every other element alone."""
    q, k, v, N, slots, pos = make(4, 4, 2, 128, 16, torch.bfloat16, 3, fused=False)
    q[1, 2, 5] = float("inf")
    k[2, 1, 70] = float("nan")
    v[3, 0, 9] = float("nan")
    slots = np.arange(4)
    kc = torch.zeros((2, 2, 16, 128), device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    qo = torch.empty_like(q)
    freq = P.pa_rotary_frequencies(128)
    P.pa_rotary_and_cache(qo, q, k, v, kc, vc, torch.tensor(slots, device="cuda"),
                          torch.tensor(pos, dtype=torch.int32, device="cuda"), freq)
    bad = ~torch.isfinite(qo)
    assert set(map(tuple, bad.nonzero().tolist())) <= {(1, 2, 5), (1, 2, 69)} and bad.any()
    bad = torch.isnan(kc)
    assert set(map(tuple, bad.nonzero().tolist())) == {(0, 1, 2, 6), (0, 1, 2, 70)}
    assert set(map(tuple, torch.isnan(vc).nonzero().tolist())) == {(0, 0, 3, 9)}


def test_bad_slot_is_flagged_and_skipped():
    q, k, v, N, slots, pos = make(5, 4, 2, 64, 16, torch.float16, 4)
    kc = torch.zeros((2, 2, 16, 64), device="cuda", dtype=torch.float16)
    vc = torch.zeros_like(kc)
    slots = torch.tensor([0, 32, 1 << 40, 31, -1], device="cuda")
    qo = torch.full((5, 4, 64), float("nan"), device="cuda", dtype=torch.float16)
    P.pa_rotary_and_cache(qo, q, k, v, kc, vc, slots, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                          P.pa_rotary_frequencies(64))
    assert P.pa_get_device_error() == 4
    assert torch.isfinite(qo).all()                              # q is turned all the same
    rows = vc.transpose(1, 2).reshape(32, 2, 64)
    assert torch.equal(rows[0], v[0]) and torch.equal(rows[31], v[3])
    assert (rows[1:31] == 0).all()


def test_refusals_of_the_binding():
    q, k, v, N, slots, pos = make(3, 4, 2, 128, 16, torch.bfloat16, 5)
    kc = torch.zeros((N, 2, 16, 128), device="cuda", dtype=torch.bfloat16)
    vc, qo = torch.zeros_like(kc), torch.empty((3, 4, 128), device="cuda", dtype=torch.bfloat16)
    st, pt = torch.tensor(slots, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda")
    f = P.pa_rotary_frequencies(128)
    good = dict(q_out=qo, q=q, k=k, v=v, k_cache=kc, v_cache=vc, slot_mapping=st, positions=pt, inv_freq=f)
    P.pa_rotary_and_cache(**good)
    for kw, err in ((dict(positions=pt.long()), TypeError), (dict(q=q.float()), TypeError),
                    (dict(q_out=qo[:2]), ValueError), (dict(v=v[:, :1]), ValueError),
                    (dict(k_cache=kc.half()), TypeError), (dict(q=q.transpose(1, 2)), ValueError),
                    (dict(q=q.cpu()), ValueError), (dict(positions=pt[:2]), ValueError),
                    (dict(inv_freq=[]), RuntimeError), (dict(q_out=k.expand(3, 2, 128)), ValueError),
                    (dict(inv_freq=np.ones((8, 8))), ValueError)):
        with pytest.raises(err):
            P.pa_rotary_and_cache(**{**good, **kw})


def test_same_as_reshape_where_nothing_turns():
    """Position 0 turns nothing: the cache is the one pa_reshape_and_cache writes, bit for bit."""
    q, k, v, N, slots, _ = make(40, 4, 4, 128, 16, torch.float16, 6, fused=False)
    st = torch.tensor(slots, device="cuda")
    a = [torch.zeros((N, 4, 16, 128), device="cuda", dtype=torch.float16) for _ in range(4)]
    qo = torch.empty_like(q)
    P.pa_rotary_and_cache(qo, q, k, v, a[0], a[1], st, torch.zeros(40, dtype=torch.int32, device="cuda"),
                          P.pa_rotary_frequencies(128))
    P.pa_reshape_and_cache(k, v, a[2], a[3], st)
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3]) and torch.equal(qo, q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_codes_are_those_of_the_plain_cache_write(dtype):
    """V's codes, and K's where nothing turns, are pa_reshape_and_cache_fp8's bit for bit: the
    fp32 quotient is the one IEEE division gives, for values over the whole range of the type
    and scales from ordinary to extreme."""
    T, Hkv, D = 512, 12, 128
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((T, Hkv, D), generator=g, device="cuda") * 8
    span = 15.0 if dtype == torch.float16 else 126.0
    x[::2] *= torch.exp2((torch.rand((T // 2, Hkv, D), generator=g, device="cuda") * 2 - 1) * span)
    x = x.to(dtype)
    x[5, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0], device="cuda")
    y = x.flip(0).contiguous()
    scale = torch.tensor([0.013, 1.0, 0.02, 3.7e-3, 448.0, 1e-20, 1e20, 2.0 ** -120, 2.0 ** 120, 1e-44, 0.0,
                          -0.5], device="cuda")
    slots = torch.randperm(T, generator=g, device="cuda")
    pools = [torch.zeros((T // 16, Hkv, 16, D), device="cuda", dtype=torch.uint8) for _ in range(4)]
    P.pa_rotary_and_cache_fp8(torch.empty_like(x), x, x, y, pools[0], pools[1], slots,
                              torch.zeros(T, dtype=torch.int32, device="cuda"), [0.0] * 64, scale, scale)
    P.pa_reshape_and_cache_fp8(x, y, pools[2], pools[3], slots, scale, scale)
    assert torch.equal(pools[1], pools[3])
    # turning by nothing leaves every finite value; an infinity meets 0 * inf = NaN
    keep = torch.isfinite(x.float()).all(-1)[slots.argsort()].view(T // 16, 16, Hkv).transpose(1, 2)
    assert torch.equal(pools[0][keep], pools[2][keep])
