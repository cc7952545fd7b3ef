"""Distance slopes up to the largest finite ones: a bias beyond fp32 leaves the nearest token
(positive slopes) or the farthest visible one (negative slopes) with all the weight."""
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import CHUNK_TOL, build, check

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


SHAPES = [(2, 1, 128, torch.float16, False), (8, 1, 64, torch.bfloat16, False),
          (16, 1, 128, torch.float16, False), (40, 1, 128, torch.bfloat16, False), (4, 1, 128, torch.float16, True),
          (8, 1, 128, torch.bfloat16, True), (16, 1, 128, torch.float16, True), (2, 1, 64, torch.bfloat16, True)]


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("slope", [1e20, 3e36, 3e38, -1e20, -3e38])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8,new", [
    (2, 2, 128, torch.float32, False, None),        # (fp32 caches have no chunk call)
    *[(*shape, new) for shape in SHAPES for new in (None, [3, 5, 2], [40, 70, 33])]])
def test_slopes_without_bound(Hq, Hkv, D, dtype, fp8, new, slope, softcap):
    lens = [200, 130, 77]
    c = build(2, lens, new or [1] * 3, Hq, Hkv, D, 16, dtype, fp8, window=60)
    slopes = torch.full((Hq,), slope, device="cuda")
    for part in (-1, 128):
        out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
        kw = dict(softcap=softcap, alibi_slopes=slopes, window=60, partition_size=part)
        if new is None:
            f = P.pa_decode_mod_fp8 if fp8 else P.pa_decode_mod
            f(out, c.q, *c.pools, c.table, c.context_lens, c.scale, Hkv, 16, **kw)
        else:
            f = P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod
            f(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, c.scale, Hkv, 16,
              max_query_len=max(new), **kw)
        torch.cuda.synchronize()
        assert P.pa_get_device_error() == 0
        rows = []
        for s, (L, n) in enumerate(zip(lens, c.new)):
            for j in range(n):
                t = L - n + j
                rows.append(c.V[s][:, t if slope > 0 else max(0, t - 59)].repeat_interleave(Hq // Hkv, 0))
        ref = torch.stack(rows).cpu().numpy()
        check(out, ref, float(abs(ref).max()), CHUNK_TOL)
