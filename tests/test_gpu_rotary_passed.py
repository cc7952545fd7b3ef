"""Dims from rotary_dim on pass unchanged, bit for bit, whatever they and their neighbours
hold: infinities, NaNs with a payload, negative zeros.  rotary_dim here ends inside a 16-byte
vector of interleaved pairs, or leaves whole vectors past it."""
import pytest
import torch

import paged_kv_cache_119_gb300 as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

BITS = {torch.float16: torch.int16, torch.bfloat16: torch.int16, torch.float32: torch.int32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_119_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def clear_error_word(built):
    P.pa_get_device_error()
    yield


def odd_rows(shape, dtype, rot, g):
    """Ordinary numbers in the turned dims; past them every third element is special."""
    x = torch.randn(shape, generator=g, device="cuda").to(dtype)
    w = x.view(BITS[dtype])
    exp = {torch.float16: 0x7c00, torch.bfloat16: 0x7f80, torch.float32: 0x7f800000}[dtype]
    sign = -0x8000 if dtype != torch.float32 else -0x80000000
    special = torch.tensor([exp, exp | sign, exp | 5, exp | sign | 9, sign, 0], device="cuda").to(w.dtype)
    tail = w[..., rot:]
    at = torch.arange(tail.numel(), device="cuda").reshape(tail.shape)
    tail.copy_(torch.where(at % 3 == 0, special[(at // 3) % len(special)], tail))
    return x


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("inter", [True, False], ids=["interleaved", "halves"])
@pytest.mark.parametrize("rot", [2, 20, 36, 64])
@pytest.mark.parametrize("D,T,Hq,Hkv", [(128, 5, 4, 2), (80, 33, 3, 3)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fp8", [False, True])
def test_passed_dims(dtype, fp8, D, T, Hq, Hkv, rot, inter, inplace):
    g = torch.Generator(device="cuda").manual_seed(rot + D)
    q, k = odd_rows((T, Hq, D), dtype, rot, g), odd_rows((T, Hkv, D), dtype, rot, g)
    v = odd_rows((T, Hkv, D), dtype, 0, g)
    N, B = T // 4 + 2, 16
    slots = torch.randperm(N * B, generator=g, device="cuda")[:T]
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    freq = P.pa_rotary_frequencies(rot)
    q0 = q.clone()
    qo = q if inplace else torch.zeros_like(q)
    pool = lambda: torch.zeros((N, Hkv, B, D), device="cuda", dtype=torch.uint8 if fp8 else dtype)
    kc, vc, kw, vw = pool(), pool(), pool(), pool()
    if fp8:
        F8 = torch.float8_e4m3fn
        ks, vs = (torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.005 for _ in range(2))
        P.pa_rotary_and_cache_fp8(qo, q, k, v, kc.view(F8), vc.view(F8), slots, pos, freq, ks, vs,
                                  interleaved=inter)
        P.pa_reshape_and_cache_fp8(k, v, kw.view(F8), vw.view(F8), slots, ks, vs)
    else:
        P.pa_rotary_and_cache(qo, q, k, v, kc, vc, slots, pos, freq, interleaved=inter)
        P.pa_reshape_and_cache(k, v, kw, vw, slots)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    bits = lambda x: x if x.dtype == torch.uint8 else x.view(BITS[dtype])
    assert torch.equal(bits(qo)[..., rot:], bits(q0)[..., rot:])
    assert torch.equal(bits(kc)[..., rot:], bits(kw)[..., rot:])
    assert torch.equal(bits(vc), bits(vw))
    assert torch.isfinite(qo[..., :rot].float()).all()
