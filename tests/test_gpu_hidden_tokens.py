"""What lies in the slots of tokens that no row sees changes no bit of a capped call: the form
of tanh is chosen from scores that rows see."""
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import FP8, build

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


def fill_hidden(c, value):
    """Copies of the pools whose NaN slots (the ones no row sees) hold `value` instead."""
    pools = []
    for x in c.pools[:2]:
        if c.fp8:
            w = x.view(torch.uint8).clone()
            code = torch.tensor(value).clamp(-448, 448).to(FP8).view(torch.uint8).item()
            pools.append(torch.where((w & 0x7f) == 0x7f, torch.full_like(w, code), w).view(FP8))
        else:
            pools.append(torch.where(x.isnan(), torch.full_like(x, value), x))
    return (*pools, *c.pools[2:])


def run(c, pools, decode, slopes, part):
    out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    kw = dict(softcap=30.0, alibi_slopes=slopes, window=c.window, global_lens=c.global_lens, partition_size=part)
    if decode:
        f = P.pa_decode_mod_fp8 if c.fp8 else P.pa_decode_mod
        f(out, c.q, *pools, c.table, c.context_lens, c.scale, c.Hkv, c.B, **kw)
    else:
        f = P.pa_chunk_attention_mod_fp8 if c.fp8 else P.pa_chunk_attention_mod
        f(out, c.q, *pools, c.table, c.context_lens, c.query_start, c.scale, c.Hkv, c.B,
          max_query_len=max(c.new), **kw)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    return out


@pytest.mark.parametrize("window,glob", [(0, 0), (37, 0), (100, 21)])
@pytest.mark.parametrize("new", [None, [3, 5, 2, 4], [40, 70, 90, 33]], ids=["decode", "few", "long"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", [
    (2, 1, 128, torch.float16, False), (4, 1, 128, torch.float16, False), (8, 1, 64, torch.bfloat16, False),
    (16, 1, 128, torch.bfloat16, False), (24, 1, 128, torch.float16, False), (40, 1, 64, torch.float16, False),
    (4, 1, 128, torch.bfloat16, True), (8, 1, 128, torch.float16, True), (16, 1, 128, torch.bfloat16, True),
    (8, 1, 64, torch.bfloat16, True)])
def test_hidden_tokens_change_nothing(Hq, Hkv, D, dtype, fp8, new, window, glob):
    lens = [130, 75, 301, 41]
    c = build(1, lens, new or [1] * 4, Hq, Hkv, D, 16, dtype, fp8, window, [glob] * 4 if glob else None)
    for slopes in (None, torch.linspace(0.01, 0.5, Hq, device="cuda")):
        for part in (-1, 128):
            want = run(c, c.pools, new is None, slopes, part)
            assert torch.isfinite(want).all()
            for value in (0.0, 300.0, -2e4):
                assert torch.equal(run(c, fill_hidden(c, value), new is None, slopes, part), want), value
