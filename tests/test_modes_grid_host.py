"""What the launch grids refuse at the C interface (no GPU: every call here returns before it
launches anything, for want of a workspace at the latest)."""
import pytest

from paged_kv_cache_119_gb300 import _native as N
from test_block_scale_host import attn_args
from test_modes_host import INV, WS, chunk_args, lib      # noqa: F401 (lib: the fixture)

# 32 heads, one a kv head: 2047 tiles of 256 rows a head fit in 65535
@pytest.mark.parametrize("rows,status", [(262016, WS), (262017, WS), (524032, WS), (524033, INV)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_long_chunks(lib, D, cap, rows, status):                          # noqa: F811
    """One length for every mode and head_dim, whatever rows a CTA takes."""
    kw = dict(max_context=1 << 20, stride=1 << 16, tokens=100, max_query=rows, part=128, Hq=32, Hkv=32, D=D, cap=cap)
    assert lib.pa_chunk_attention_mod(*chunk_args(**kw).values()) == status


@pytest.mark.parametrize("group,rows,status", [(3, 1 << 17, WS), (3, 85 * 4095, WS), (3, 85 * 4095 + 1, INV),
                                               (100, 2 * 4095, WS), (100, 2 * 4095 + 1, INV)])
def test_long_chunks_of_a_group(lib, group, rows, status):                # noqa: F811
    """256 / group tokens a tile: 16 kv heads of 4095 tiles."""
    kw = dict(max_context=1 << 20, stride=1 << 16, tokens=100, max_query=rows, part=128, Hq=16 * group, Hkv=16, D=64)
    assert lib.pa_chunk_attention_mod(*chunk_args(**kw).values()) == status


@pytest.mark.parametrize("fn,D", [("pa_cross_attention", 64), ("pa_cross_attention", 128),
                                  ("pa_cross_attention_fp8", 128), ("pa_cross_attention_fp8_block", 128)])
def test_long_cross_rows(lib, fn, D):                                     # noqa: F811
    for rows, status in ((262017, WS), (524032, WS), (524033, INV)):
        kw = dict(mq=rows, rows=100, max_ctx=4096, bt_stride=256, Hq=32, Hkv=32, D=D, part=128)
        if fn.endswith("block"):
            kw["stride"] = 32
        assert getattr(lib, fn)(*attn_args(fn, **kw)) == status


def test_row_mode_grids_end_at_65535(lib):                                # noqa: F811
    """E4M3 caches at head_dim 64 run on a decode kernel's row mode, whose grid has its tiles in y."""
    fn = "pa_cross_attention_fp8_block"
    kw = dict(rows=100, max_ctx=4096, bt_stride=256, Hq=32, Hkv=32, D=64, stride=32, part=128)
    assert lib.pa_cross_attention_fp8_block(*attn_args(fn, mq=2047 * 64, **kw)) == WS
    assert lib.pa_cross_attention_fp8_block(*attn_args(fn, mq=2047 * 64 + 1, **kw)) == INV
