"""The chunk kernel's last wave, cut into parts and merged, in the forms of block-scaled caches and of
cross attention: units of one CTA each, a few more than there are SMs, against the definition in 64
bits (tolerances in test_gpu_block_scale.py).  Empty contexts, contexts shorter than their rows and
sequences without rows lie among the whole units and the cut ones.
"""
import pytest
import torch

import block_reference as R
from test_gpu_block_scale import check, no_error

pytestmark = pytest.mark.gpu
HEADS = 8
FORMS = [("chunk", "block", 128, 16, torch.bfloat16), ("chunk", "block", 128, 32, torch.float16),
         ("chunk", "half", 64, 16, torch.bfloat16), ("chunk", "half", 64, 32, torch.float16),
         ("cross", "block", 128, 16, torch.bfloat16), ("cross", "block", 128, 32, torch.float16),
         ("cross", "head", 128, 16, torch.bfloat16), ("cross", "half", 128, 16, torch.bfloat16),
         ("cross", "half", 64, 16, torch.float16), ("cross", "half", 64, 32, torch.bfloat16)]


def build(call, kind, D, B, dtype):
    """One row tile a sequence and head.  The last three sequences' 24 units are the cut ones."""
    S = torch.cuda.get_device_properties(0).multi_processor_count // HEADS + 3
    # (16-bit caches at head_dim 64 have CTAs of one row tile, which are not cut, but for long contexts
    # and full tiles)
    full = kind == "half" and D == 64
    new = [256 if full else 40 - i % 5 for i in range(S)]
    lens = [(2100 if full else 1040) + 7 * i % 260 for i in range(S)]
    if not full:
        new[4] = 0
    for s, L in ((1, 0), (2, 11), (S - 3, 0), (S - 1, 9)):
        lens[s] = L if call == "cross" else max(new) + L      # (a chunk's context holds its rows)
    return R.build(81, lens, new, HEADS, HEADS, D, B, dtype, causal=call == "chunk", kind=kind)


def run(c, call, kind, **kw):
    """The output, and whether the call was cut: a part wrote to the workspace."""
    import paged_kv_cache_119_gb300 as pa
    fn = {"chunk block": pa.pa_chunk_attention_fp8_block, "chunk half": pa.pa_chunk_attention_mod,
          "cross block": pa.pa_cross_attention_fp8_block, "cross head": pa.pa_cross_attention_fp8,
          "cross half": pa.pa_cross_attention}[f"{call} {kind}"]
    most = max(c.lens)
    ws = torch.full((pa.pa_chunk_workspace_bytes(c.q.shape[0], HEADS, c.D, most),), 0x5a, dtype=torch.uint8,
                    device="cuda")
    out = torch.full(c.q.shape, float("nan"), device="cuda")
    fn(out, c.q, *c.args, c.query_start, c.scale, HEADS, c.B, max_query_len=max(c.new), max_context_len=most,
       workspace=ws, **kw)
    return out, bool((ws != 0x5a).any())


@pytest.mark.parametrize("call,kind,D,B,dtype", FORMS)
def test_last_wave(call, kind, D, B, dtype):
    c = build(call, kind, D, B, dtype)
    ref, size = R.attend(c)
    out, cut = run(c, call, kind)
    assert cut
    check(out, ref, size)
    whole, cut = run(c, call, kind, partition_size=-1)
    assert not cut
    check(whole, ref, size)
    if call == "cross":
        for s in (1, len(c.lens) - 3):
            at = int(c.query_start[s])
            assert (out[at:at + c.new[s]] == 0).all()
    assert no_error()


@pytest.mark.parametrize("call,kind,D,B,dtype", FORMS)
def test_bad_sequences(call, kind, D, B, dtype):
    """Lengths out of range and blocks outside the pool, among the whole units and the cut ones:
    their rows become NaN, all others stay as they are."""
    import paged_kv_cache_119_gb300 as pa
    from paged_kv_cache_119_gb300 import _native as N
    c = build(call, kind, D, B, dtype)
    good, _ = run(c, call, kind)
    start = c.query_start.tolist()
    most, S = max(c.lens), len(c.lens)
    for s, L in ((0, most + 1), (5, -1), (S - 1, -7), (S - 2, most + 1)):
        keep = c.lens[s]
        c.context_lens[s] = L
        out, _ = run(c, call, kind)
        c.context_lens[s] = keep
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == N.PA_DEVERR_CONTEXT_LEN
        rows = torch.zeros(out.shape[0], dtype=torch.bool)
        rows[start[s]:start[s + 1]] = True
        assert torch.isnan(out[rows]).all() and torch.equal(out[~rows], good[~rows])
    for s in (3, S - 2):
        keep = int(c.table[s, 20])
        c.table[s, 20] = c.pools[0].shape[0]
        out, _ = run(c, call, kind)
        c.table[s, 20] = keep
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == N.PA_DEVERR_BLOCK_ID
        rows = torch.zeros(out.shape[0], dtype=torch.bool)
        rows[start[s]:start[s + 1]] = True
        assert torch.isnan(out[rows]).all() and torch.equal(out[~rows], good[~rows])
