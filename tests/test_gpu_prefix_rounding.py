"""The shared-prefix decode keeps the accuracy and the range of pa_decode whatever the size of
the group: probabilities of wide groups are not one 16-bit term, and V is not converted."""
import numpy as np
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import FP8, ROWS_TOL, build, check, reference

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("members", [2, 5, 40, 130])
@pytest.mark.parametrize("D,B,dtype,fp8", [(128, 16, torch.bfloat16, False), (128, 32, torch.float16, False),
                                           (64, 16, torch.bfloat16, False), (64, 32, torch.float16, False),
                                           (128, 16, torch.bfloat16, True), (128, 32, torch.float16, True)])
def test_two_tokens(D, B, dtype, fp8, members):
    """Two tokens carry the weight, 1 and w = 2^(-a log2 e), a row's own a in (0, 4), with V 0
    and 1: the output is w / (1 + w).  Each score is one product, and a step of it (2^-24 of
    at most 4, times the softmax scale's and log2 e's roundings) moves the output by less
    than 4 2^-22; exp2 is good to 2^-22; two 16-bit terms of a weight are within 2^-16 of it
    (bf16: half a step of each, 2^-9 twice) and enter with w / (1 + w)^2 <= 1/4; the other
    tokens weigh less than 200 e^-50.  So 2^-17 bounds the error.  One f16 term is off by up
    to 2^-11 / 4 = 2^-13."""
    G, P0 = 4, 128
    rng = np.random.default_rng(members)
    q = torch.zeros((members, G, D), device="cuda")
    a = torch.tensor(rng.uniform(0.05, 4.0, (members, G)), device="cuda")
    q[..., 0] = a.float()
    q[..., 1] = 64.0
    q = q.to(dtype)
    a = q[..., 0].double()
    N = P0 // B + 1
    k, v = (torch.zeros((N, 1, B, D), device="cuda") for _ in range(2))
    k[..., 1] = -1.0                                  # every token: -64
    k[0, 0, 3, 1] = k[-2, 0, 5, 1] = 0.0              # but two
    k[-2, 0, 5, 0] = -1.0
    v[-2, 0, 5] = 1.0
    table = i32([list(range(N))] * members)
    lens = i32([P0 + s % 3 for s in range(members)])
    out = torch.zeros((members, G, D), device="cuda")
    args = (table, lens, i32([P0] * members), i32([0, members]), 1.0, 1, B)
    kw = dict(max_group_size=members, max_prefix_len=P0, max_suffix_len=2)
    if fp8:
        one = torch.ones(1, device="cuda")
        P.pa_decode_prefix_fp8(out, q, k.to(FP8), v.to(FP8), one, one, *args, **kw)
    else:
        P.pa_decode_prefix(out, q, k.to(dtype), v.to(dtype), *args, **kw)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    w = torch.exp(-a)
    err = (out.double() - (w / (1 + w))[..., None]).abs().max().item()
    assert err <= 2.0 ** -17, err


@pytest.mark.parametrize("power", [40, -40])
@pytest.mark.parametrize("members", [3, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_values_beyond_the_range_of_f16(D, members, power):
    """A bf16 cache whose V is 2^40 or 2^-40 times the usual: the bound grows alike."""
    c = build(5, [96 + s % 7 for s in range(members)], [1] * members, 8, 2, D, 16, torch.bfloat16,
              shared=[(0, members, 96)])
    c.v_cache *= 2.0 ** power
    c.V = [v * 2.0 ** power for v in c.V]
    out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    P.pa_decode_prefix(out, c.q, *c.pools, c.table, c.context_lens, torch.tensor(c.shared_len, device="cuda"),
                       i32([0, members]), c.scale, c.Hkv, c.B, max_group_size=members, max_prefix_len=96,
                       max_suffix_len=6)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    ref, vmax = reference(c)
    check(out, ref, vmax, ROWS_TOL + 2.0 ** -16)
