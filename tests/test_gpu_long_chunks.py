"""Chunks whose kv heads x row tiles pass 65535: bounds alone, and rows in earnest.  Tolerances as in
attn_reference.py."""
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import CHUNK_TOL, build, check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("window", [0, 30])
def test_a_loose_bound(D, dtype, window):
    c = build(61, [140, 75], [100, 60], 32, 32, D, 16, dtype, window=window)
    table = torch.full((2, 40000), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    out = torch.full(c.q.shape, float("nan"), device="cuda")
    P.pa_chunk_attention_mod(out, c.q, *c.pools, table, c.context_lens, c.query_start, c.scale, 32, 16,
                             max_query_len=500000, window=window)
    check(out, *reference(c), CHUNK_TOL)
    assert P.pa_get_device_error() == 0


def test_rows_past_65535_tiles():
    """270 000 rows of 32 heads under a window of 64, against rows picked among them."""
    n, H, D, B, window = 270000, 32, 64, 16, 64
    g = torch.Generator(device="cuda").manual_seed(62)
    N = (n + B - 1) // B
    table = torch.randperm(N, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    k, v = (torch.randn((N, H, B, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    q = torch.randn((n, H, D), generator=g, device="cuda", dtype=torch.float16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    P.pa_chunk_attention_mod(out, q, k, v, table, lens, start, D ** -0.5, H, B, max_query_len=n, window=window,
                             partition_size=-1)             # (a workspace for any cut would not fit)
    assert P.pa_get_device_error() == 0
    rows = torch.cat([torch.arange(0, 70), torch.randint(0, n, (200,), generator=torch.Generator().manual_seed(63)),
                      torch.arange(n - 200, n)]).cuda()
    t = rows[:, None] - torch.arange(window - 1, -1, -1, device="cuda")[None]        # [R, window]
    at = t.clamp(min=0)
    K, V = (x[table[0, at // B].long(), :, at % B].double() for x in (k, v))         # [R, window, H, D]
    x = torch.einsum("rhd,rthd->rht", q[rows].double(), K) * D ** -0.5
    p = torch.softmax(x.masked_fill((t < 0)[:, None], float("-inf")), -1)
    ref = torch.einsum("rht,rthd->rhd", p, V)
    check(out[rows], ref.cpu().numpy(), float(v.abs().max()), CHUNK_TOL)
    assert torch.isfinite(out).all()
