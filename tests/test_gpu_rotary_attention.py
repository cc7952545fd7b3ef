"""The rotary cache write and the attention calls as a serving step runs them together, and
the calls' use of memory: captured graphs, a shared workspace, pools and contexts beyond 32
bits.  References are 64-bit over what the cache holds; tolerances are attn_reference.py's
(CHUNK_TOL wherever a pass may take the tcgen05 kernel)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_119_gb300 as P
from attn_reference import CHUNK_TOL, ROWS_TOL, build, check

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


def gathered(pool, scale, blocks, tokens, fp8):
    """[Hkv, tokens, D] in 64 bits: what the cache holds in these blocks."""
    x = pool[torch.as_tensor(blocks, device="cuda").long()]
    x = x.view(torch.float8_e4m3fn).float().double() if fp8 else x.double()
    if fp8:
        x = x * scale.double()[:, None, None]
    return x.transpose(0, 1).reshape(pool.shape[1], -1, pool.shape[3])[:, :tokens]


def attend(q, K, V, scale, pos, softcap=0.0, window=0, glob=0):
    """Rows q [n, Hq, D] at positions pos [n] over K, V [Hkv, L, D], all in 64 bits."""
    n, Hq, D = q.shape
    G = Hq // K.shape[0]
    x = torch.einsum("nhgd,htd->hngt", q.double().view(n, -1, G, D), K) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    t = torch.arange(K.shape[1], device="cuda")[None]
    at = torch.as_tensor(pos, device="cuda")[:, None]
    sees = t <= at
    if window:
        sees &= at - t < window
    sees |= t < glob
    p = torch.softmax(x.masked_fill(~sees[None, :, None], float("-inf")), -1)
    return torch.einsum("hngt,htd->nhgd", p, V).reshape(n, Hq, D).cpu().numpy()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (4, 4, 64, 32), (24, 2, 128, 16)])
def test_prompt_then_forked_decode(Hq, Hkv, D, B, fp8):
    """A prompt is written and attended in one chunk, then forked into five continuations whose
    steps (rotary write, shared-prefix decode, capped and windowed decode) are one captured
    graph with one workspace; a padded row (slot -1, no tokens) rides along."""
    dtype, S, shared, steps = torch.bfloat16, 6, 3 * 32, 4
    g = torch.Generator(device="cuda").manual_seed(Hq + B)
    rng = np.random.default_rng(Hq + D)
    need = shared // B + 1                                   # blocks of a continuation's row
    N = shared // B + S + 2
    ids = rng.permutation(N)
    table = np.zeros((S, need), dtype=np.int32)
    table[:, :-1] = ids[:shared // B]
    table[:, -1] = ids[shared // B:shared // B + S]
    raw = torch.uint8 if fp8 else dtype
    kc, vc = (torch.full((N, Hkv, B, D), 0x7f if fp8 else float("nan"), dtype=raw, device="cuda") for _ in range(2))
    ks, vs = (torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.01 for _ in range(2))
    scales = (ks, vs) if fp8 else ()
    freq = P.pa_rotary_frequencies(D, scaling="linear", factor=2.0)
    scale = D ** -0.5
    rotary = P.pa_rotary_and_cache_fp8 if fp8 else P.pa_rotary_and_cache
    prefix = P.pa_decode_prefix_fp8 if fp8 else P.pa_decode_prefix
    mod = P.pa_decode_mod_fp8 if fp8 else P.pa_decode_mod
    chunk = P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod

    def projection(T):
        x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dtype)
        return [t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1)]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    # the prompt: its first 20 tokens see one another
    q, k, v = projection(shared)
    slots = torch.tensor([int(ids[t // B]) * B + t % B for t in range(shared)], device="cuda")
    qr = torch.empty((shared, Hq, D), dtype=dtype, device="cuda")
    rotary(qr, q, k, v, kc, vc, slots, i32(list(range(shared))), freq, *scales)
    out = torch.empty_like(qr)
    chunk(out, qr, kc, vc, *scales, i32(table[:1]), i32([shared]), i32([0, shared]), scale, Hkv, B,
          max_query_len=shared, softcap=20.0, global_lens=i32([20]), max_global_len=32)
    K, V = (gathered(c, s, ids[:shared // B], shared, fp8) for c, s in ((kc, ks), (vc, vs)))
    check(out, attend(qr, K, V, scale, np.arange(shared), softcap=20.0, glob=20), V.abs().max().item(), CHUNK_TOL)

    # the steps
    W, tb = 40, i32(table)
    q, k, v = projection(S)
    qr, o1, o2 = (torch.empty((S, Hq, D), dtype=dtype, device="cuda") for _ in range(3))
    pos, slots = i32([0] * S), torch.full((S,), -1, dtype=torch.int64, device="cuda")
    lens, plens, start = i32([shared] * (S - 1) + [0]), i32([shared] * (S - 1) + [0]), i32([0, S - 1, S])
    most = shared + B
    ws = torch.empty(max(P.pa_decode_prefix_workspace_bytes(S, Hq, D, shared, B),
                         P.pa_decode_workspace_bytes(S, Hq, D, most, B)), dtype=torch.uint8, device="cuda")

    def step():
        rotary(qr, q, k, v, kc, vc, slots, pos, freq, *scales)
        prefix(o1, qr, kc, vc, *scales, tb, lens, plens, start, scale, Hkv, B, max_group_size=S - 1,
               max_prefix_len=shared, max_suffix_len=B, workspace=ws)
        mod(o2, qr, kc, vc, *scales, tb, lens, scale, Hkv, B, softcap=5.0, window=W, max_context_len=most,
            workspace=ws)

    step()                                                   # no new token yet
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(steps):
        for dst, src in zip((q, k, v), projection(S)):
            dst.copy_(src)
        at = shared + n
        pos.copy_(i32([at] * (S - 1) + [0]))
        slots.copy_(torch.tensor([int(b) * B + n for b in table[:S - 1, -1]] + [-1]))
        lens.copy_(i32([at + 1] * (S - 1) + [0]))
        graph.replay()
        torch.cuda.synchronize()
        assert P.pa_get_device_error() == 0
        assert not o1[-1].any() and not o2[-1].any()         # the padded row
        for s in range(S - 1):
            K, V = (gathered(c, sc, table[s], at + 1, fp8) for c, sc in ((kc, ks), (vc, vs)))
            vmax = V.abs().max().item()
            check(o1[s:s + 1], attend(qr[s:s + 1], K, V, scale, [at]), vmax, CHUNK_TOL)
            check(o2[s:s + 1], attend(qr[s:s + 1], K, V, scale, [at], softcap=5.0, window=W), vmax, ROWS_TOL)


def test_two_graphs_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn on one stream, an eager call
    between them: each gives what it gives alone."""
    c = build(5, [1500, 1400, 2300], [1] * 3, 8, 1, 128, 16, torch.float16, shared=[(0, 2, 1024)])
    plens, start = torch.tensor(c.shared_len, device="cuda"), torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    need = max(P.pa_decode_prefix_workspace_bytes(3, 8, 128, 1024, 2304), P.pa_decode_workspace_bytes(3, 8, 128, 2304, 16))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(c.q) for _ in range(3)]
    q2 = c.q * 0.5

    def a():
        P.pa_decode_prefix(outs[0], c.q, *c.pools, c.table, c.context_lens, plens, start, c.scale, 1, 16,
                           max_group_size=2, max_prefix_len=1024, max_suffix_len=2304, workspace=ws)

    def b():
        P.pa_decode_mod(outs[1], q2, *c.pools, c.table, c.context_lens, c.scale, 1, 16, softcap=9.0,
                        max_context_len=2304, workspace=ws)

    def e():
        P.pa_decode_mod(outs[2], c.q, *c.pools, c.table, c.context_lens, c.scale, 1, 16, window=700,
                        max_context_len=2304, workspace=ws)

    want = []
    for f, o in zip((a, b, e), outs):
        f()
        torch.cuda.synchronize()
        want.append(o.clone())
    graphs = []
    for f in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for o in outs:
        o.fill_(float("nan"))
    for _ in range(20):
        graphs[0].replay()
        graphs[1].replay()
        e()
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_calls_on_two_streams_at_once():
    """Calls in flight together, each with its own workspace and output."""
    c = build(6, [2600, 900, 1700, 64], [1] * 4, 8, 2, 128, 32, torch.bfloat16, shared=[(0, 3, 512)])
    plens, start = torch.tensor(c.shared_len, device="cuda"), torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")

    def call(i, out, stream):
        if i % 2:
            P.pa_decode_mod(out, c.q, *c.pools, c.table, c.context_lens, c.scale, 2, 32, softcap=30.0, window=900,
                            stream=stream)
        else:
            P.pa_decode_prefix(out, c.q, *c.pools, c.table, c.context_lens, plens, start, c.scale, 2, 32,
                               max_group_size=3, max_prefix_len=512, stream=stream)

    want = []
    for i in range(2):
        want.append(torch.empty_like(c.q))
        call(i, want[-1], None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(c.q) for _ in range(16)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        call(i, o, streams[i % 4] if i % 3 else streams[i % 4].cuda_stream)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


@pytest.mark.parametrize("Hq,Hkv,dtype,fp8", [(8, 8, torch.float16, False), (64, 8, torch.bfloat16, False),
                                              (16, 8, torch.float16, True), (64, 8, torch.bfloat16, True)])
def test_pools_beyond_32_bits(Hq, Hkv, dtype, fp8):
    """A pool of more than 2^32 elements: rows written to, and read from, its last blocks."""
    B, D, T = 16, 128, 200
    N = (1 << 32) // (Hkv * B * D) + 40
    raw = torch.uint8 if fp8 else dtype
    kc, vc = (torch.empty((N, Hkv, B, D), dtype=raw, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)
    n = (T + B - 1) // B
    blocks = [N - 1 - 2 * i for i in range(n)]
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    slots = torch.tensor([blocks[t // B] * B + t % B for t in range(T)], device="cuda")
    ks, vs = (torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.01 for _ in range(2))
    scales = (ks, vs) if fp8 else ()
    kc[blocks], vc[blocks] = 0, 0
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rotary = P.pa_rotary_and_cache_fp8 if fp8 else P.pa_rotary_and_cache
    qr = torch.empty_like(q)
    rotary(qr, q, k, v, kc, vc, slots, pos, P.pa_rotary_frequencies(D), *scales)
    K, V = (gathered(c, s, blocks, T, fp8) for c, s in ((kc, ks), (vc, vs)))
    assert fp8 or torch.equal(V.to(dtype), v.transpose(0, 1))
    tb = torch.tensor([blocks], dtype=torch.int32, device="cuda")
    one = torch.tensor([T], dtype=torch.int32, device="cuda")
    vmax, scale = V.abs().max().item(), D ** -0.5
    out = torch.empty((1, Hq, D), dtype=torch.float32, device="cuda")
    (P.pa_decode_mod_fp8 if fp8 else P.pa_decode_mod)(
        out, qr[-1:], kc, vc, *scales, tb, one, scale, Hkv, B, window=90, softcap=30.0)
    check(out, attend(qr[-1:], K, V, scale, [T - 1], softcap=30.0, window=90), vmax, ROWS_TOL)
    (P.pa_decode_prefix_fp8 if fp8 else P.pa_decode_prefix)(
        out, qr[-1:], kc, vc, *scales, tb, one, torch.tensor([160], dtype=torch.int32, device="cuda"),
        torch.tensor([0, 1], dtype=torch.int32, device="cuda"), scale, Hkv, B, max_group_size=1, max_prefix_len=160)
    check(out, attend(qr[-1:], K, V, scale, [T - 1]), vmax, CHUNK_TOL)
    rows = torch.empty((90, Hq, D), dtype=torch.float32, device="cuda")
    (P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod)(
        rows, qr[-90:], kc, vc, *scales, tb, one, torch.tensor([0, 90], dtype=torch.int32, device="cuda"), scale,
        Hkv, B, max_query_len=90, softcap=30.0)
    check(rows, attend(qr[-90:], K, V, scale, np.arange(T - 90, T), softcap=30.0), vmax, CHUNK_TOL)
    torch.cuda.synchronize()
    assert P.pa_get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,dtype,fp8", [(2, 2, torch.float16, False), (4, 1, torch.bfloat16, False),
                                              (16, 1, torch.float16, False), (2, 2, torch.float16, True),
                                              (16, 1, torch.bfloat16, True)])
def test_the_longest_context(Hq, Hkv, dtype, fp8):
    """A window and a few first tokens of a context of almost 2^30 tokens."""
    B, D, L, W, glob = 16, 128, (1 << 30) - 5, 100, 21
    lo = (L - 70 - W) // B                                   # first block either call looks at
    head, tail = (glob + B - 1) // B, (L + B - 1) // B - lo
    g = torch.Generator(device="cuda").manual_seed(4)
    x = [torch.randn((head + tail, Hkv, B, D), generator=g, device="cuda") for _ in range(2)]
    ks, vs = (torch.full((Hkv,), 1.0 / 64, device="cuda") for _ in range(2))
    kc, vc = ((t * 64).to(torch.float8_e4m3fn) if fp8 else t.to(dtype) for t in x)
    scales = (ks, vs) if fp8 else ()
    table = torch.full((1, (1 << 30) // B), -1, dtype=torch.int32, device="cuda")
    table[0, :head] = torch.arange(head)
    table[0, lo:lo + tail] = torch.arange(head, head + tail)
    K, V = (gathered(c.view(torch.uint8) if fp8 else c, s, list(range(head + tail)), (head + tail) * B, fp8)
            for c, s in ((kc, ks), (vc, vs)))
    where = np.concatenate([np.arange(head * B), np.arange(lo * B, (lo + tail) * B)])     # positions of K's rows
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    gl = torch.tensor([glob], dtype=torch.int32, device="cuda")
    vmax, scale = V.abs().max().item(), D ** -0.5

    def want(q, pos):
        n = q.shape[0]
        y = torch.einsum("nhgd,htd->hngt", q.double().view(n, Hkv, -1, D), K) * scale
        sees = (where[None] < glob) | ((where[None] <= pos[:, None]) & (pos[:, None] - where[None] < W))
        p = torch.softmax(y.masked_fill(~torch.tensor(sees, device="cuda")[None, :, None], float("-inf")), -1)
        return torch.einsum("hngt,htd->nhgd", p, V).reshape(n, Hq, D).cpu().numpy()

    for n in (1, 3, 60):
        q = torch.randn((n, Hq, D), generator=g, device="cuda").to(dtype)
        out = torch.empty((n, Hq, D), dtype=torch.float32, device="cuda")
        kw = dict(window=W, global_lens=gl, max_global_len=glob, max_context_len=L)
        if n == 1:
            (P.pa_decode_mod_fp8 if fp8 else P.pa_decode_mod)(out, q, kc, vc, *scales, table, lens, scale, Hkv, B, **kw)
        else:
            (P.pa_chunk_attention_mod_fp8 if fp8 else P.pa_chunk_attention_mod)(
                out, q, kc, vc, *scales, table, lens, torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale,
                Hkv, B, max_query_len=n, **kw)
        torch.cuda.synchronize()
        assert P.pa_get_device_error() == 0
        check(out, want(q, np.arange(L - n, L)), vmax, ROWS_TOL if n == 1 else CHUNK_TOL)
