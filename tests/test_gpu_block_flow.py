"""The block-scaled cache as a server uses it: chunked prompts, a fork with copy-on-write of codes
and scales, decode steps beside cross attention to an encoder's states, captured and replayed, on
other streams, and swapped out and in.

Attention is compared with the definition in 64 bits over the values that the pools hold
(tolerances in test_gpu_block_scale), the pools with the appended rows: a value is within half an
E4M3 step of its row's element, 2^-4 of it or 2^-10 of the scale, and one more such rounding for
each time its block was restated (only below 2^-6 of the scale).
"""
import numpy as np
import pytest
import torch

import block_reference as R
from test_gpu_block_scale import check

pytestmark = pytest.mark.gpu
HQ, HKV, D, B = 8, 2, 128, 16
SCALE = D ** -0.5
FREQ = 10000.0 ** (-2.0 * np.arange(D // 2) / D)


class Pool:
    def __init__(self, blocks, dtype):
        self.k, self.v = (torch.full((blocks, HKV, B, D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((blocks, 4), float("nan"), device="cuda") for _ in range(2))
        self.dtype = dtype

    @property
    def args(self):
        return self.k, self.v, self.ks, self.vs

    def dense(self, row, L):
        """K and V of a table row's first L tokens, in 64 bits."""
        ids = torch.as_tensor(row[:(L + B - 1) // B]).long()
        return [(R.decode(p[ids.cuda()]) * s[ids.cuda(), :HKV].double().cpu()[:, :, None, None]).transpose(0, 1)
                .reshape(HKV, -1, D)[:, :L] for p, s in ((self.k, self.ks), (self.v, self.vs))]


def reference(pool, table, lens, new, q, causal=True):
    c = R.Case()
    c.lens, c.new, c.Hq, c.Hkv, c.D, c.causal, c.scale, c.q = lens, new, HQ, HKV, D, causal, SCALE, q
    kv = [pool.dense(t, L) for t, L in zip(table, lens)]
    c.K, c.V = [x[0] for x in kv], [x[1] for x in kv]
    return R.attend(c)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rows(g, n, dtype):
    x = torch.randn((n, HQ + 2 * HKV, D), device="cuda", generator=g)
    x *= torch.exp2(torch.randn((n, 1, 1), device="cuda", generator=g))
    x = x.to(dtype)
    return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompts_fork_steps_cross_and_swap(dtype):
    import paged_kv_cache_119_gb300 as pa
    g = torch.Generator(device="cuda").manual_seed(41)
    pool = Pool(40, dtype)
    ids = np.random.default_rng(41).permutation(40).astype(np.int32)
    free = list(ids)
    table = np.full((3, 8), -1, dtype=np.int32)
    lens = [0, 0]
    history = [[], []]
    # ---- two prompts in chunks: rotate and append, then attend
    for step in ([40, 7], [30, 21], [3, 0]):
        for s, n in enumerate(step):
            for b in range((lens[s] + B - 1) // B, (lens[s] + n + B - 1) // B):
                table[s, b] = free.pop()
            lens[s] += n
        q, k, v = rows(g, sum(step), dtype)
        start = np.concatenate([[0], np.cumsum(step)])
        for s in range(2):
            history[s].append(v[start[s]:start[s + 1]])
        qr = torch.empty((sum(step), HQ, D), dtype=dtype, device="cuda")
        bt, cl, qs = ints(table[:2]), ints(lens), ints(start)
        pa.pa_rotary_and_append_fp8_block(qr, q, k, v, *pool.args, bt, cl, qs, FREQ, max_query_len=max(step))
        out = torch.empty_like(qr)
        pa.pa_chunk_attention_fp8_block(out, qr, *pool.args, bt, cl, qs, SCALE, HKV, B, max_query_len=max(step))
        check(out, *reference(pool, table, lens, step, qr))
    for s in range(2):
        told = pool.dense(table[s], lens[s])[1]
        true = torch.cat(history[s]).double().cpu().transpose(0, 1)
        scale = pool.vs[torch.tensor(table[s][:(lens[s] + B - 1) // B]).long().cuda()][:, :HKV].double().cpu()
        scale = scale.repeat_interleave(B, 0)[:lens[s]].T[:, :, None]
        assert ((told - true).abs() <= true.abs() * 2.0 ** -4 + 3 * 2.0 ** -10 * scale).all()
    # ---- sequence 0 forks: its full blocks are shared, the last one copied with its scales
    table[2] = table[0]
    last = (lens[0] - 1) // B
    assert lens[0] % B
    table[2, last] = free.pop()
    pair = [(int(table[0, last]), int(table[2, last]))]
    pa.pa_copy_blocks(pool.k, pool.v, pair)
    pa.pa_copy_blocks(pool.ks, pool.vs, pair)
    lens.append(lens[0])
    # ---- an encoder's states, appended as they are
    enc = Pool(20, dtype)
    enc_lens, enc_rows = [70, 33, 70], 70 + 33
    enc_table = np.full((3, 5), -1, dtype=np.int32)
    enc_table[0], enc_table[1, :3], enc_table[2] = np.arange(5), [7, 5, 6], np.arange(5)
    _, ek, ev = rows(g, enc_rows, dtype)
    pa.pa_append_fp8_block(ek, ev, *enc.args, ints(enc_table[:2]), ints(enc_lens[:2]), ints([0, 70, 103]),
                           max_query_len=70)
    # ---- decode steps of all three beside cross attention, eager and then captured
    bt, cl, qs = ints(table), ints(lens), ints([0, 1, 2, 3])
    ebt, ecl = ints(enc_table), ints(enc_lens)
    q, k, v = (torch.empty((3, h, D), dtype=dtype, device="cuda") for h in (HQ, HKV, HKV))
    qr, out, crossed = (torch.empty((3, HQ, D), dtype=dtype, device="cuda") for _ in range(3))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        pa.pa_rotary_and_append_fp8_block(qr, q, k, v, *pool.args, bt, cl, qs, FREQ, max_query_len=1)
        pa.pa_decode_fp8_block(out, qr, *pool.args, bt, cl, SCALE, HKV, B, workspace=ws)
        pa.pa_cross_attention_fp8_block(crossed, qr, *enc.args, ebt, ecl, qs, SCALE, HKV, B, max_query_len=1,
                                        workspace=ws)

    graph = None
    for t in range(20):
        for s in range(3):
            if lens[s] % B == 0:
                table[s, lens[s] // B] = free.pop()
            lens[s] += 1
        for dst, src in zip((q, k, v), rows(g, 3, dtype)):
            dst.copy_(src)
        bt.copy_(ints(table))
        cl.copy_(ints(lens))
        if t == 3:
            keep = [x.clone() for x in pool.args]
            step()
            eager = out.clone(), crossed.clone(), [x.clone() for x in pool.args]
            for x, y in zip(pool.args, keep):
                x.copy_(y)
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        if graph is None:
            step()
        else:
            graph.replay()
        if t == 3:
            assert torch.equal(out, eager[0]) and torch.equal(crossed, eager[1])
            assert all(torch.equal(a[:, :HKV] if a.dtype == torch.float32 else a,
                                   b[:, :HKV] if b.dtype == torch.float32 else b)
                       for a, b in zip([x.nan_to_num(7.0) if x.dtype == torch.float32 else x for x in pool.args],
                                       [x.nan_to_num(7.0) if x.dtype == torch.float32 else x for x in eager[2]]))
        check(out, *reference(pool, table, lens, [1] * 3, qr))
        check(crossed, *reference(enc, enc_table, enc_lens, [1] * 3, qr, causal=False))
    # ---- the fork shares what it had and not what came after
    assert table[0, 0] == table[2, 0] and not torch.equal(out[0], out[2])
    # ---- out to pinned memory and back into other blocks
    used = sorted({int(b) for s in range(3) for b in table[s] if b >= 0})
    host = [torch.empty((40, *x.shape[1:]), dtype=x.dtype).pin_memory() for x in pool.args]
    back = [b for b in range(40) if b not in used][:len(used)]
    back += used[:len(used) - len(back)]
    before = out.clone()
    for group in (slice(0, 2), slice(2, 4)):
        pa.pa_swap_blocks(list(pool.args[group]), host[group], [(b, i) for i, b in enumerate(used)])
    torch.cuda.synchronize()
    for x in pool.args:
        x.fill_(0x7f if x.dtype == torch.uint8 else float("nan"))
    for group in (slice(0, 2), slice(2, 4)):
        pa.pa_swap_blocks(host[group], list(pool.args[group]), [(i, b) for i, b in enumerate(back)])
    move = dict(zip(used, back))
    bt.copy_(ints([[move.get(int(b), -1) for b in row] for row in table]))
    pa.pa_decode_fp8_block(out, qr, *pool.args, bt, cl, SCALE, HKV, B, workspace=ws)
    assert torch.equal(out, before)
    assert pa.pa_get_device_error() == 0


def test_other_streams_and_two_calls_at_once():
    """Calls on streams of their own, side by side, each with a workspace of its own."""
    import paged_kv_cache_119_gb300 as pa
    cases = [R.build(50 + i, [700, 300, 513], [n] * 3, 8, 2, 128, 16, torch.bfloat16, causal=i % 2 == 0)
             for i, n in enumerate((1, 3, 40, 70))]

    def call(c, out, stream=None):
        fn = pa.pa_chunk_attention_fp8_block if c.causal else pa.pa_cross_attention_fp8_block
        if c.causal and c.new[0] == 1:
            return pa.pa_decode_fp8_block(out, c.q, *c.args, c.scale, c.Hkv, c.B, stream=stream)
        return fn(out, c.q, *c.args, c.query_start, c.scale, c.Hkv, c.B, max_query_len=c.new[0], stream=stream)

    want = [call(c, torch.empty_like(c.q)).clone() for c in cases]
    torch.cuda.synchronize()
    for how in ("with", "argument"):
        streams = [torch.cuda.Stream() for _ in cases]
        outs = [torch.full_like(c.q, float("nan")) for c in cases]
        torch.cuda.synchronize()
        for _ in range(5):
            for c, o, s in zip(cases, outs, streams):
                if how == "with":
                    with torch.cuda.stream(s):
                        call(c, o)
                else:
                    call(c, o, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_a_cache_of_another_device_is_refused():
    import paged_kv_cache_119_gb300 as pa
    c = R.build(60, [30], [1], 2, 2, 128, 16, torch.bfloat16)
    out = torch.empty_like(c.q)
    for i in range(6):
        args = list(c.args)
        args[i] = args[i].cpu()
        with pytest.raises(ValueError):
            pa.pa_decode_fp8_block(out, c.q, *args, c.scale, 2, 16)
    with pytest.raises(ValueError):
        pa.pa_decode_fp8_block(out, c.q, *c.args, c.scale, 2, 16, workspace=torch.empty(10))


def test_padded_batch():
    """Sequences without rows, and a batch padded to a captured size with empty ones."""
    import paged_kv_cache_119_gb300 as pa
    c = R.build(61, [40, 0, 90, 0], [3, 0, 5, 0], 8, 2, 128, 16, torch.bfloat16)
    ref, size = R.attend(c)
    out = torch.empty_like(c.q)
    check(pa.pa_chunk_attention_fp8_block(out, c.q, *c.args, c.query_start, c.scale, 2, 16, max_query_len=5), ref,
          size)
    k = torch.randn((8, 2, 128), device="cuda").bfloat16()
    before = [x.clone().view(torch.uint8) for x in (*c.pools, *c.scales)]
    pa.pa_append_fp8_block(k, k, *c.pools, *c.scales, c.table, c.context_lens, c.query_start, max_query_len=5)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    touched = {int(c.table_np[0, 2]), int(c.table_np[2, 5])}
    for x, y in zip((*c.pools, *c.scales), before):
        same = (x.view(torch.uint8) == y).flatten(1).all(1).cpu()
        assert {int(i) for i in torch.nonzero(~same)} <= touched
