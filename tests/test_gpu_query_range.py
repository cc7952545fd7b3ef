"""bf16 queries far from 1 over E4M3 caches: the modified-score and shared-prefix calls scale
each query row into f16's range by a power of two, both ways, so that its 8-bit mantissas
convert exactly.  The K scale makes up for it here, and the scores are those of ordinary
rows: the tolerance is the usual one (attn_reference.py)."""
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


def scaled(c, power, heads):
    """Query heads `heads` times 2^power, K times 2^-power (both exact)."""
    c.q[:, heads] *= 2.0 ** power
    c.k_scale *= 2.0 ** -power
    c.K = [k * 2.0 ** -power for k in c.K]
    return c


def attend(c, kind):
    out = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    if kind == "decode":
        P.pa_decode_mod_fp8(out, c.q, *c.pools, c.table, c.context_lens, c.scale, c.Hkv, c.B)
    elif kind == "prefix":
        S = len(c.lens)
        P.pa_decode_prefix_fp8(out, c.q, *c.pools, c.table, c.context_lens,
                               torch.tensor(c.shared_len, device="cuda"),
                               torch.tensor([0, S], dtype=torch.int32, device="cuda"), c.scale, c.Hkv, c.B,
                               max_group_size=S, max_prefix_len=int(c.shared_len[0]), max_suffix_len=200)
    else:
        P.pa_chunk_attention_mod_fp8(out, c.q, *c.pools, c.table, c.context_lens, c.query_start, c.scale,
                                     c.Hkv, c.B, max_query_len=max(c.new))
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    return out


KINDS = ["decode", "prefix", "few", "long"]


def case(kind, Hq, D):
    shared = [(0, 4, 64)] if kind == "prefix" else None
    new = {"few": [3, 5, 2, 4], "long": [50, 60, 40, 33]}.get(kind, [1] * 4)
    return build(1, [100, 75, 201, 90], new, Hq, 1, D, 16, torch.bfloat16, True, shared=shared)


@pytest.mark.parametrize("power", [-40, -20, 30])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,D", [(1, 128), (4, 128), (8, 128), (16, 128), (40, 128), (2, 64), (8, 64)])
def test_rows_far_from_one(Hq, D, kind, power):
    c = scaled(case(kind, Hq, D), power, slice(None))
    ref, vmax = reference(c)
    check(attend(c, kind), ref, vmax, CHUNK_TOL)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,D", [(4, 128), (8, 128), (16, 128), (40, 128), (8, 64)])
def test_small_rows_beside_large_ones(Hq, D, kind):
    """Odd heads are 2^-34 of the even ones, whose scores are beyond any tolerance and are not
    looked at: a row's scale is its own."""
    c = scaled(case(kind, Hq, D), -34, slice(1, None, 2))
    ref, vmax = reference(c)
    check(attend(c, kind)[:, 1::2], ref[:, 1::2], vmax, CHUNK_TOL)
