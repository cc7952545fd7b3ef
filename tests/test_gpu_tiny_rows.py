"""bf16 rows far below 1 over E4M3 caches whose K scales are as small: their scores are 0 to any
weight, in tiles with hidden tokens too, so a row is the mean of the V rows that it sees.

The tolerance is that of test_gpu_block_scale.py; the references take the rows as they are.
"""
import pytest
import torch

import block_reference as R
from test_gpu_block_scale import check, no_error

pytestmark = pytest.mark.gpu

LENS, NEW = [100, 70, 200], [50, 40, 64]


def tiny(c, power):
    """Every other token's rows times 2^power (exact in bf16)."""
    c.q[::2] *= 2.0 ** power
    return c


@pytest.mark.parametrize("call", ["chunk", "cross"])
@pytest.mark.parametrize("power", [-115, -100, -85])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 4, 128), (8, 1, 64)])
def test_a_block_of_zero_keys(call, power, B, Hq, Hkv, D):
    """What an append of zeros leaves: codes of 0 and the least scale, here in the last tile."""
    import paged_kv_cache_119_gb300 as pa
    c = tiny(R.build(51, LENS, NEW, Hq, Hkv, D, B, torch.bfloat16, causal=call == "chunk"), power)
    for s, L in enumerate(LENS):
        lb = (L - 1) // B - 1                     # the last whole block
        blk = int(c.table_np[s, lb])
        c.pools[0].view(torch.uint8)[blk] = 0
        c.scales[0][blk] = 2.0 ** -48
        c.K[s][:, lb * B:lb * B + B] = 0
    ref, size = R.attend(c)
    fn = pa.pa_chunk_attention_fp8_block if call == "chunk" else pa.pa_cross_attention_fp8_block
    for part in (0, 128):
        out = torch.empty(c.q.shape, device="cuda")
        fn(out, c.q, *c.args, c.query_start, c.scale, Hkv, B, max_query_len=max(NEW), partition_size=part)
        check(out, ref, size)
    assert no_error()


@pytest.mark.parametrize("call", ["plain", "mod", "window", "cross"])
@pytest.mark.parametrize("power", [-115, -100, -85])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 4, 128), (8, 1, 64)])
def test_a_tiny_scale_a_head(call, power, Hq, Hkv, D):
    import paged_kv_cache_119_gb300 as pa
    c = tiny(R.build(52, LENS, NEW, Hq, Hkv, D, 16, torch.bfloat16, causal=call != "cross", kind="head"), power)
    for s in range(len(LENS)):
        c.K[s] *= 2.0 ** -48 / c.scales[0].double().cpu()[:, None, None]
    c.scales[0].fill_(2.0 ** -48)
    ref, size = R.attend(c)
    fn = {"plain": pa.pa_chunk_attention_fp8, "cross": pa.pa_cross_attention_fp8}.get(call, pa.pa_chunk_attention_mod_fp8)
    kw = dict(window=1000) if call == "window" else {}
    out = torch.empty(c.q.shape, device="cuda")
    fn(out, c.q, *c.args, c.query_start, c.scale, Hkv, 16, max_query_len=max(NEW), **kw)
    check(out, ref, size)
    assert no_error()
