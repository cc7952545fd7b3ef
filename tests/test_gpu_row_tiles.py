"""16-bit caches at head_dim 64, where a CTA of the chunk kernel takes one row tile or two: shapes on
either side of the rules that choose and that cut contexts, against the definition in 64 bits
(tolerances in test_gpu_block_scale.py)."""
import pytest
import torch

import block_reference as R
from test_gpu_block_scale import check, no_error

pytestmark = pytest.mark.gpu


def call(c, L):
    """The output, and whether contexts were cut: a part wrote to the workspace."""
    import paged_kv_cache_119_gb300 as pa
    out = torch.full(c.q.shape, float("nan"), device="cuda")
    ws = torch.full((pa.pa_chunk_workspace_bytes(c.q.shape[0], c.Hq, c.D, L) + 16,), 0x5a, dtype=torch.uint8,
                    device="cuda")
    fn = pa.pa_chunk_attention_mod if c.causal else pa.pa_cross_attention
    fn(out, c.q, *c.args, c.query_start, c.scale, c.Hkv, c.B, max_query_len=max(c.new), max_context_len=L,
       workspace=ws)
    return out, bool((ws != 0x5a).any())


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# (sequences, new tokens, ragged, context, query heads, kv heads), whether it is cut on 152 SMs
SHAPES = {
    "one tile of rows": ((6, 70, True, 500, 8, 8), False),
    "an SM for each of two tiles": ((10, 200, True, 600, 8, 8), False),
    "three tiles of rows": ((4, 300, True, 900, 8, 4), False),
    "short contexts, full tiles": ((30, 256, False, 700, 8, 8), False),
    "long contexts, full tiles": ((24, 256, False, 2100, 8, 8), True),
    "long contexts, ragged rows": ((24, 256, True, 2100, 8, 8), False),
    "few units over a long context": ((2, 64, True, 9000, 8, 4), True),
    "few units of full tiles over a longer one": ((1, 64, False, 17000, 8, 2), True),
    "an SM each, a context worth a cut": ((12, 40, True, 4200, 8, 8), True),
    "an SM each, a context too short for a cut": ((12, 40, True, 1900, 8, 8), False),
    "a group that does not divide the tile": ((5, 100, True, 800, 9, 3), True),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,B", [(torch.float16, 32), (torch.bfloat16, 16)])
@pytest.mark.parametrize("shape", SHAPES)
def test_forms(shape, dtype, B, causal):
    (S, n, ragged, L, Hq, Hkv), cut = SHAPES[shape]
    new = [n - (11 * i) % (n // 2) if ragged else n for i in range(S)]
    lens = [max(m, L - 13 * i) for i, m in enumerate(new)]
    if not causal and S > 1:
        lens[1], lens[S - 1] = 0, 7
    c = R.build(91, lens, new, Hq, Hkv, 64, B, dtype, causal=causal, kind="half")
    ref, size = R.attend(c)
    out, was_cut = call(c, L)
    check(out, ref, size)
    assert no_error()
    assert was_cut == cut or sms() != 152
