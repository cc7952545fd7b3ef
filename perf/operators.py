"""Cases of the rotary cache write, the shared-prefix decode and the attention with modified
scores: their inputs, a plain form of each in elementary torch operations, the calls of the
library, and the definition in 64 bits.

Every case works on a paged cache: pools [blocks][kv heads][block_size][head_dim], int32
block tables, int64 slots.  Pools are full of values (a pool in use holds stale tokens in
every free slot), and table entries past a sequence's last block are 0.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
#: what the pools hold: the type of the queries, or one-byte codes
FP8 = torch.float8_e4m3fn


# --------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a small batch: four new tokens, latency alone
        dict(name="rotary_step4", op="rotary", tokens=4, hq=32, hkv=8, d=128, b=16, dtype="bf16", fp8=False,
             rot=128, inter=False, scaling="none", pos=32768),
        # the cache write of a chunked prefill of 8 prompts, 512 tokens each, with
        # interleaved pairs and frequencies stretched for long contexts
        dict(name="rotary_prefill4096", op="rotary", tokens=4096, hq=64, hkv=8, d=128, b=16, dtype="bf16",
             fp8=False, rot=128, inter=True, scaling="by_parts", pos=131072),
        # long prompts into an E4M3 cache, half of each head rotated, an odd token count
        dict(name="rotary_fp8_16391", op="rotary", tokens=16391, hq=32, hkv=32, d=128, b=32, dtype="f16",
             fp8=True, rot=64, inter=False, scaling="linear", pos=65536),
        # two short conversations forked from one system prompt: latency
        dict(name="prefix_2x3", op="prefix", groups=2, members=3, prefix=256, suffix=40, hq=32, hkv=8, d=128,
             b=16, dtype="bf16", fp8=False),
        # few-shot prompts: 16 groups of 8 sequences over 1024 shared tokens
        dict(name="prefix_16x8", op="prefix", groups=16, members=8, prefix=1024, suffix=256, hq=32, hkv=8,
             d=128, b=16, dtype="bf16", fp8=False),
        # one long document asked about by many: 96 sequences over 16384 shared tokens
        dict(name="prefix_1x96_long", op="prefix", groups=1, members=96, prefix=16384, suffix=384, hq=64,
             hkv=8, d=128, b=16, dtype="bf16", fp8=False),
        # the same use over an E4M3 cache
        dict(name="prefix_fp8_4x32", op="prefix", groups=4, members=32, prefix=4096, suffix=300, hq=32, hkv=8,
             d=128, b=32, dtype="bf16", fp8=True),
        # a batch of mixed lengths with distance-biased scores, one query head per kv head
        dict(name="mod_decode_alibi", op="decode", seqs=64, ctx=2048, spread=True, hq=40, hkv=40, d=128, b=16,
             dtype="f16", fp8=False, cap=0.0, slopes=True, window=0, keep=0),
        # long contexts with capped scores, eight query heads per kv head
        dict(name="mod_decode_cap_long", op="decode", seqs=8, ctx=32768, spread=False, hq=64, hkv=8, d=128,
             b=16, dtype="bf16", fp8=False, cap=50.0, slopes=False, window=0, keep=0),
        # sliding window that keeps the first tokens, E4M3 cache: reads 4160 of ~16384 tokens
        dict(name="mod_decode_window_fp8", op="decode", seqs=48, ctx=16384, spread=False, hq=64, hkv=8, d=128,
             b=32, dtype="bf16", fp8=True, cap=0.0, slopes=False, window=4096, keep=64),
        # checking five speculated tokens per sequence, capped and windowed
        dict(name="mod_chunk_verify5", op="chunk", seqs=32, new=5, ctx=1500, hq=32, hkv=8, d=128, b=16,
             dtype="f16", fp8=False, cap=30.0, slopes=False, window=1024, keep=0),
        # a chunked prefill with capped scores
        dict(name="mod_chunk_prefill", op="chunk", seqs=4, new=512, ctx=8192, hq=64, hkv=8, d=128, b=16,
             dtype="bf16", fp8=False, cap=50.0, slopes=False, window=0, keep=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "prefix", "decode", "chunk"])
    fp8 = rng.random() < 0.3
    dtype = rng.choice(["bf16", "bf16", "f16"])
    hkv, g = rng.choice([(8, 4), (8, 8), (16, 1), (32, 1), (4, 7), (10, 4), (8, 2)])
    base = dict(op=op, hq=hkv * g, hkv=hkv, b=rng.choice([16, 32]), dtype=dtype, fp8=fp8)
    if op == "rotary":
        d = rng.choice([64, 128])
        if not fp8 and rng.random() < 0.15:
            base["dtype"] = "f32"
        return dict(base, tokens=_log(rng, 1, 8000), d=d, rot=rng.choice([d, d, d // 2, d // 4 + 4]),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                    pos=_log(rng, 1000, 1000000))
    if op == "prefix":
        members = _log(rng, 1, 96)
        groups = _log(rng, 1, max(1, 128 // members))
        most = min(8192, 1000000 // (groups * hkv), 12000000 // (groups * members * hkv))
        return dict(base, d=128 if fp8 else rng.choice([64, 128, 128]), groups=groups, members=members,
                    prefix=32 * _log(rng, 1, most // 32), suffix=_log(rng, 1, 600))
    mods = dict(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.4,
                window=rng.choice([0, 0, 1, _log(rng, 16, 4096)]), keep=0)
    if mods["window"] and rng.random() < 0.5:
        mods["keep"] = _log(rng, 1, 200)
    if op == "decode":
        seqs = _log(rng, 1, 128)
        return dict(base, d=rng.choice([64, 128, 128]), seqs=seqs, ctx=_log(rng, 1, min(16384, 2000000 // (seqs * hkv))),
                    spread=rng.random() < 0.6, **mods)
    seqs = _log(rng, 1, 16)
    new = _log(rng, 2, 512 if seqs <= 4 else 100)
    if rng.random() < 0.25:   # a prompt whose first tokens see one another
        mods["keep"] = _log(rng, 1, new)
    return dict(base, d=128 if fp8 else rng.choice([64, 128, 128]), seqs=seqs, new=new,
                ctx=new + _log(rng, 1, 32768 // seqs - 600), **mods)


# --------------------------------------------------------------------------- the inputs

def _lens(case, rng):
    """Context length of each sequence (the new tokens counted)."""
    if case["op"] == "prefix":
        return [case["prefix"] + int(x) for x in rng.integers(1, case["suffix"] + 1, case["groups"] * case["members"])]
    if case["op"] == "chunk":
        return [int(x) for x in rng.integers(max(case["new"], case["ctx"] * 7 // 8), case["ctx"] + 1, case["seqs"])]
    low = 1 if case["spread"] else max(1, case["ctx"] * 15 // 16)
    return [int(x) for x in rng.integers(low, case["ctx"] + 1, case["seqs"])]


def _new(case, seqs):
    """New tokens of each sequence of a chunk case: all but the first a little ragged."""
    return [case["new"] - (37 * i) % max(1, case["new"] // 8) for i in range(seqs)]


def _pool(g, blocks, case, std):
    x = torch.empty((blocks, case["hkv"], case["b"], case["d"]), device="cuda", dtype=DTYPES[case["dtype"]])
    x.normal_(0.0, std, generator=g)
    return x


def _rotary_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, hq, hkv, d, b = (case[k] for k in ("tokens", "hq", "hkv", "d", "b"))
    dt = DTYPES[case["dtype"]]
    # the rows of one projection: q, k and v of a token lie beside each other
    qkv = torch.empty((t, (hq + 2 * hkv) * d), device="cuda", dtype=dt).normal_(0.0, 1.0, generator=g)
    blocks = max(1, math.ceil(1.1 * t / b))
    slots = rng.permutation(blocks * b)[:t]
    if t > 8:
        slots[t // 2] = -1                       # padding of a captured step
    positions = rng.integers(0, case["pos"], t)
    half = case["rot"] // 2
    s = dict(case=case, q=qkv[:, :hq * d].unflatten(1, (hq, d)),
             k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
             v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
             slots=torch.tensor(slots, dtype=torch.int64, device="cuda"),
             positions=torch.tensor(positions, dtype=torch.int32, device="cuda"),
             freq=_frequencies(case["rot"], case["scaling"]),
             magnitude=1.0 + 0.1 * math.log(8.0) if case["scaling"] == "by_parts" else 1.0)
    assert s["freq"].shape == (half,)
    s["freq_gpu"] = torch.tensor(s["freq"], device="cuda")
    shape = (blocks, hkv, b, d)
    if case["fp8"]:
        s["k_cache"] = torch.zeros(shape, device="cuda", dtype=FP8)
        s["v_cache"] = torch.zeros(shape, device="cuda", dtype=FP8)
        s["k_scale"] = torch.tensor(rng.uniform(0.01, 0.03, hkv), dtype=torch.float32, device="cuda")
        s["v_scale"] = torch.tensor(rng.uniform(0.01, 0.03, hkv), dtype=torch.float32, device="cuda")
    else:
        s["k_cache"] = torch.zeros(shape, device="cuda", dtype=dt)
        s["v_cache"] = torch.zeros(shape, device="cuda", dtype=dt)
    return s


def _frequencies(rot, scaling):
    """Radians per position of each pair, base 10000, stretched for contexts 8 times as long."""
    i = np.arange(rot // 2, dtype=np.float64)
    factor = 8.0
    if scaling == "ntk" and rot > 2:
        return (10000.0 * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return keep * f + (1.0 - keep) * f / factor
    return f


def _attention_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, hq, hkv, d = (case[k] for k in ("b", "hq", "hkv", "d"))
    lens = _lens(case, rng)
    s_count = len(lens)
    need = [math.ceil(n / b) for n in lens]
    shared = case["prefix"] // b if case["op"] == "prefix" else 0
    fresh = sum(n - shared for n in need) + (shared * case["groups"] if shared else 0)
    blocks = math.ceil(1.05 * fresh) + 1
    ids = rng.permutation(blocks)
    table = np.zeros((s_count, max(need)), dtype=np.int32)
    at = 0
    for s in range(s_count):
        if shared and s % case["members"] == 0:
            common = ids[at:at + shared]
            at += shared
        if shared:
            table[s, :shared] = common
        own_blocks = need[s] - shared
        table[s, shared:need[s]] = ids[at:at + own_blocks]
        at += own_blocks
    new = _new(case, s_count) if case["op"] == "chunk" else [1] * s_count
    rows = sum(new)
    dt = DTYPES[case["dtype"]]
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              table=torch.tensor(table, device="cuda"), max_len=max(lens), max_new=max(new), scale=d ** -0.5)
    # scores of a few units, as trained attention has them
    st["q"] = torch.empty((rows, hq, d), device="cuda", dtype=dt).normal_(0.0, 3.0, generator=g)
    k, v = _pool(g, blocks, case, 1.0), _pool(g, blocks, case, 1.0)
    if case["fp8"]:
        st["k_scale"] = torch.tensor(rng.uniform(0.008, 0.02, hkv), dtype=torch.float32, device="cuda")
        st["v_scale"] = torch.tensor(rng.uniform(0.008, 0.02, hkv), dtype=torch.float32, device="cuda")
        k = (k / st["k_scale"][:, None, None]).clamp_(-448, 448).to(FP8)
        v = (v / st["v_scale"][:, None, None]).clamp_(-448, 448).to(FP8)
    st["k_cache"], st["v_cache"] = k, v
    start = np.concatenate([[0], np.cumsum(new)])
    st["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    if case["op"] == "prefix":
        st["shared"] = torch.full((s_count,), case["prefix"], dtype=torch.int32, device="cuda")
        st["group_start"] = torch.arange(0, s_count + 1, case["members"], dtype=torch.int32, device="cuda")
        return st
    # a row of the padded batch [sequence][new token] and back
    seq = np.repeat(np.arange(s_count), new)
    tok = np.concatenate([np.arange(n) for n in new])
    st["seq"] = torch.tensor(seq, device="cuda")
    st["tok"] = torch.tensor(tok, device="cuda")
    st["pos"] = torch.tensor(np.asarray(lens)[seq] - np.asarray(new)[seq] + tok, device="cuda")
    st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32,
                                device="cuda") if case["slopes"] else None
    st["keep"] = torch.tensor(np.minimum(case["keep"], lens), dtype=torch.int32, device="cuda") \
        if case["keep"] else None
    return st


def prepare(case, seed):
    return _rotary_inputs(case, seed) if case["op"] == "rotary" else _attention_inputs(case, seed)


# --------------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rotary(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["freq_gpu"]
    cos = (torch.cos(angle) * s["magnitude"]).float()
    sin = (torch.sin(angle) * s["magnitude"]).float()
    q = _rotate(s["q"], cos, sin, case["rot"], case["inter"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, case["rot"], case["inter"])
    v = s["v"]
    if case["fp8"]:
        k = (k / s["k_scale"][:, None]).clamp(-448, 448).to(FP8)
        v = (v.float() / s["v_scale"][:, None]).clamp(-448, 448).to(FP8)
    else:
        k = k.to(s["q"].dtype)
    live = s["slots"] >= 0
    slots = s["slots"][live]
    blk, off = slots // case["b"], slots % case["b"]
    if case["fp8"]:
        s["k_cache"].view(torch.uint8)[blk, :, off] = k.view(torch.uint8)[live]
        s["v_cache"].view(torch.uint8)[blk, :, off] = v.view(torch.uint8)[live]
    else:
        s["k_cache"][blk, :, off] = k[live]
        s["v_cache"][blk, :, off] = v[live]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gather(cache, table, scale):
    """[S, Hkv, W * B, D] in 32 bits."""
    s, w = table.shape
    x = cache.view(torch.uint8)[table.long()].view(FP8) if scale is not None else cache[table.long()]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
    case = s["case"]
    group = case["hq"] // case["hkv"]
    k = _gather(s["k_cache"], s["table"], s.get("k_scale"))
    v = _gather(s["v_cache"], s["table"], s.get("v_scale"))
    t = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"].long()
    count, n = lens.numel(), s["max_new"]
    if case["op"] == "chunk":
        q = torch.zeros((count, n, case["hq"], case["d"]), device="cuda")
        pos = torch.zeros((count, n), dtype=torch.int64, device="cuda")
        q[s["seq"], s["tok"]] = s["q"].float()
        pos[s["seq"], s["tok"]] = s["pos"]
    else:
        q, pos = s["q"].float()[:, None], lens[:, None] - 1
    # rows [S, Hkv, n * G]: q . k for every row and token
    rows = q.unflatten(2, (case["hkv"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(rows * s["scale"], k.transpose(2, 3)).unflatten(2, (n, group))
    visible = t <= pos[:, :, None]
    if case["op"] != "prefix":
        gap = pos[:, :, None] - t
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        if s["slopes"] is not None:
            slope = s["slopes"].view(case["hkv"], 1, group, 1)
            x = x - slope * gap.abs()[:, None, :, None, :].float()
        if case["window"]:
            visible = visible & (gap < case["window"])
        if s["keep"] is not None:
            visible = visible | (t < s["keep"].long()[:, None, None])
    x = x.masked_fill(~visible[:, None, :, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o = o[s["seq"], s["tok"]] if case["op"] == "chunk" else o[:, 0]
    return o.to(s["q"].dtype)


# --------------------------------------------------------------------------- the library

def _own_rotary(s):
    import paged_kv_cache_119_gb300 as pa
    case = s["case"]
    q = torch.empty((case["tokens"], case["hq"], case["d"]), device="cuda", dtype=s["q"].dtype)
    args = (q, s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["freq"])
    if case["fp8"]:
        pa.pa_rotary_and_cache_fp8(*args, s["k_scale"], s["v_scale"], interleaved=case["inter"],
                                   magnitude=s["magnitude"])
    else:
        pa.pa_rotary_and_cache(*args, interleaved=case["inter"], magnitude=s["magnitude"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import paged_kv_cache_119_gb300 as pa
    case = s["case"]
    out = torch.empty_like(s["q"])
    pools = (out, s["q"], s["k_cache"], s["v_cache"])
    if case["fp8"]:
        pools += (s["k_scale"], s["v_scale"])
    if case["op"] == "prefix":
        call = pa.pa_decode_prefix_fp8 if case["fp8"] else pa.pa_decode_prefix
        return call(*pools, s["table"], s["lens"], s["shared"], s["group_start"], s["scale"], case["hkv"], case["b"],
                    max_group_size=case["members"], max_prefix_len=case["prefix"], max_suffix_len=case["suffix"])
    mods = dict(softcap=case["cap"], alibi_slopes=s["slopes"], window=case["window"], global_lens=s["keep"],
                max_global_len=case["keep"], max_context_len=s["max_len"])
    if case["op"] == "chunk":
        call = pa.pa_chunk_attention_mod_fp8 if case["fp8"] else pa.pa_chunk_attention_mod
        return call(*pools, s["table"], s["lens"], s["start"], s["scale"], case["hkv"], case["b"],
                    max_query_len=s["max_new"], **mods)
    call = pa.pa_decode_mod_fp8 if case["fp8"] else pa.pa_decode_mod
    return call(*pools, s["table"], s["lens"], s["scale"], case["hkv"], case["b"], **mods)


def run(state):
    if state["case"]["op"] == "rotary":
        return _own_rotary(state) if own else _plain_rotary(state)
    return _own_attention(state) if own else _plain_attention(state)


# --------------------------------------------------------------------------- work

def _visible(case, length, new):
    """(tokens that some row sees, (row, token) pairs) of a sequence with `new` query tokens."""
    window = case.get("window", 0) or length
    keep = min(case.get("keep", 0), length)
    first = length - new
    pairs = 0
    for pos in range(first, length):
        low = max(0, pos - window + 1)
        pairs += (pos + 1 - low) + (min(keep, low) + max(0, keep - (pos + 1)) if keep else 0)
    low = max(0, first - window + 1)
    return (length - low) + min(keep, low), pairs


def work(case):
    esz = 4 if case["dtype"] == "f32" else 2
    ksz = 1 if case["fp8"] else esz
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        t = case["tokens"]
        return {"bytes": t * d * (2 * hq * esz + 2 * hkv * (esz + ksz)) + 12 * t,
                "flops": t * (hq + hkv) * case["rot"] * 3}
    token = 2 * hkv * d * ksz
    if case["op"] == "prefix":
        count = case["groups"] * case["members"]
        tail = count * (case["suffix"] + 1) / 2
        return {"bytes": (case["groups"] * case["prefix"] + tail) * token + 2 * count * hq * d * esz,
                "flops": 4.0 * d * hq * (count * case["prefix"] + tail)}
    if case["op"] == "chunk":
        length, new, count = case["ctx"] * 15 // 16, case["new"], case["seqs"]
        length = max(length, new)
    else:
        length = (case["ctx"] + 1) // 2 if case["spread"] else case["ctx"] * 31 // 32
        length, new, count = max(1, length), 1, case["seqs"]
    seen, pairs = _visible(case, length, new)
    return {"bytes": count * (seen * token + 2 * new * hq * d * esz), "flops": 4.0 * d * hq * count * pairs}


# --------------------------------------------------------------------------- in 64 bits

def _exact_rotary(case, s):
    out = {}
    angle = torch.outer(s["positions"].double(), torch.tensor(s["freq"], device="cuda"))
    turn = torch.polar(torch.full_like(angle, s["magnitude"]), angle)           # m e^(i angle)
    half = case["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    pools = {}
    for name in ("k", "v"):
        pool = s[name + "_cache"].double()
        x = out["k"] if name == "k" else s["v"].double()
        if case["fp8"]:
            x = x / s[name + "_scale"].double()[:, None]
        flat = pool.transpose(1, 2).reshape(-1, case["hkv"], case["d"])         # [slot][head][dim]
        live = s["slots"] >= 0
        flat = flat.index_copy(0, s["slots"][live], x[live])
        pools[name + "_cache"] = flat.view(-1, case["b"], case["hkv"], case["d"]).transpose(1, 2).contiguous()
    return {"q": out["q"], **pools}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    b, hkv, d = case["b"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    start = s["start"].tolist()
    result = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        ids = s["table"][i, :(length + b - 1) // b].long()
        kv = []
        for name in ("k", "v"):
            pool = s[name + "_cache"]
            x = pool.view(torch.uint8)[ids].view(FP8) if case["fp8"] else pool[ids]
            x = x.double().transpose(0, 1).reshape(hkv, -1, d)[:, :length]
            kv.append(x * s[name + "_scale"].double()[:, None, None] if case["fp8"] else x)
        q = s["q"][start[i]:start[i + 1]].double()
        n = q.shape[0]
        at = torch.arange(length - n, length, device="cuda")[:, None]
        t = torch.arange(length, device="cuda")[None, :]
        hidden = t > at
        if case.get("window"):
            hidden = hidden | (t <= at - case["window"])
        if case.get("keep"):
            hidden = hidden & (t >= case["keep"])
        for h in range(hkv):
            x = torch.einsum("ngd,td->ngt", q[:, h * group:(h + 1) * group], kv[0][h]) * s["scale"]
            if case.get("cap"):
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case.get("slopes"):
                x = x - s["slopes"][h * group:(h + 1) * group].double()[None, :, None] * (at - t).abs()[:, None, :]
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            result[start[i]:start[i + 1], h * group:(h + 1) * group] = torch.einsum(
                "ngt,td->ngd", torch.softmax(x, dim=-1), kv[1][h])
    return result
