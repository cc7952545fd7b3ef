"""Cases of the E4M3 cache with a scale for each block and head (its write, decode and chunk
attention) and of cross attention over a paged cache: their inputs, a plain form of each in
elementary torch operations, the calls of the library, and the definition in 64 bits.

Every case works on a paged cache: pools [blocks][kv heads][block_size][head_dim] with int32
block tables.  A block-scaled pool stands for code * scale[block][head]; its scales are rows of
[blocks][stride] with the stride a multiple of four, so that they can be copied like blocks.
Pools are full of values (a pool in use holds stale tokens in every free slot), and table
entries past a sequence's last block are 0.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
FP8 = torch.float8_e4m3fn
#: the powers of two a scale is held within
LOW, HIGH = -48, 48


# --------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a small batch: a new token each, latency alone
        dict(name="append_step4", op="append", seqs=4, new=1, old=900, hq=32, hkv=8, d=128, b=16, dtype="bf16",
             rot=128, inter=False),
        # one decode step of a large batch of a multi-head model
        dict(name="append_step256", op="append", seqs=256, new=1, old=2048, hq=40, hkv=40, d=128, b=16,
             dtype="bf16", rot=128, inter=False),
        # a chunked prefill of ragged prompts, half of each head rotated in interleaved pairs
        dict(name="append_prefill", op="append", seqs=32, new=543, old=4000, hq=64, hkv=8, d=128, b=16,
             dtype="bf16", rot=64, inter=True),
        # the states of an encoder: no positions, every block opened by the call
        dict(name="append_states", op="append", seqs=24, new=1500, old=0, hq=16, hkv=16, d=64, b=32, dtype="f16",
             rot=0, inter=False),
        # a small interactive batch
        dict(name="decode_small", op="decode", seqs=4, ctx=700, spread=True, hq=32, hkv=8, d=128, b=16,
             dtype="bf16"),
        # a batch of mixed lengths, one query head per kv head
        dict(name="decode_mixed", op="decode", seqs=256, ctx=1031, spread=True, hq=40, hkv=40, d=128, b=16,
             dtype="bf16"),
        # long contexts, eight query heads per kv head
        dict(name="decode_long", op="decode", seqs=8, ctx=32768, spread=False, hq=64, hkv=8, d=128, b=16,
             dtype="bf16"),
        # checking four speculated tokens per sequence
        dict(name="chunk_verify4", op="chunk", seqs=32, new=4, ctx=1500, hq=32, hkv=8, d=128, b=16, dtype="f16"),
        # a chunked prefill
        dict(name="chunk_prefill", op="chunk", seqs=4, new=512, ctx=8192, hq=64, hkv=8, d=128, b=32,
             dtype="bf16"),
        # five beams of eight utterances, each over its encoder's states, in 16 bits
        dict(name="cross_beams", op="cross", seqs=8, new=5, ctx=1500, hq=16, hkv=16, d=64, b=16, dtype="f16",
             kind="half"),
        # prompts longer than some of the encoders' states they look at, in 16 bits
        dict(name="cross_prompts", op="cross", seqs=24, new=448, ctx=1500, hq=20, hkv=20, d=64, b=16,
             dtype="bf16", kind="half"),
        # text over the states of images, in block-scaled codes
        dict(name="cross_images", op="cross", seqs=4, new=600, ctx=6404, hq=64, hkv=8, d=128, b=16,
             dtype="bf16", kind="block"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "decode", "chunk", "cross"])
    hkv, g = rng.choice([(8, 4), (8, 8), (16, 1), (32, 1), (4, 7), (10, 4), (8, 2), (2, 16)])
    base = dict(op=op, hq=hkv * g, hkv=hkv, b=rng.choice([16, 32]), dtype=rng.choice(["bf16", "bf16", "f16"]),
                d=rng.choice([64, 128, 128]))
    if op == "append":
        seqs = _log(rng, 1, 256)
        new = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 2, 16000 // seqs)])
        d = base["d"]
        return dict(base, seqs=seqs, new=new, old=rng.choice([0, _log(rng, 1, 2000)]),
                    rot=rng.choice([d, d, d // 2, d // 4 + 4, 0]), inter=rng.random() < 0.5)
    if op == "decode":
        seqs = _log(rng, 1, 128)
        return dict(base, seqs=seqs, ctx=_log(rng, 1, min(16384, 2000000 // (seqs * hkv))),
                    spread=rng.random() < 0.6)
    seqs = _log(rng, 1, 16)
    if op == "chunk":
        new = _log(rng, 2, 512 if seqs <= 4 else 100)
        if base["d"] == 64:
            new = min(new, 64)
        return dict(base, seqs=seqs, new=new, ctx=new + _log(rng, 1, 32768 // seqs - 600))
    kind = rng.choice(["half", "head", "block", "block"])
    if kind != "half":
        base["d"] = 128
    return dict(base, seqs=seqs, new=_log(rng, 1, 600 if seqs <= 4 else 100), ctx=_log(rng, 1, 16384 // seqs),
                kind=kind)


# --------------------------------------------------------------------------- the inputs

def _pow2(e):
    """2^e as fp32, by its bits (e an int tensor)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_for(amax):
    """The smallest power of two s within [2^LOW, 2^HIGH] with amax <= 448 s."""
    m, e = torch.frexp(amax.float())                  # 448 = 0.875 * 2^9
    return _pow2(torch.where(amax > 0, e - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH))


def _spread(g, shape, std):
    """Values whose size differs from block to block and head to head, as those of a real cache do."""
    size = torch.empty((shape[0], shape[1], 1, 1), device="cuda").normal_(0.0, 0.7, generator=g)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g) * torch.exp2(size)


def _block_pool(g, blocks, case, std):
    """(codes, scales) of a block-scaled pool."""
    x = _spread(g, (blocks, case["hkv"], case["b"], case["d"]), std)
    s = _scale_for(x.abs().amax((2, 3)))
    scales = torch.ones((blocks, (case["hkv"] + 3) // 4 * 4), device="cuda")
    scales[:, :case["hkv"]] = s
    return (x / s[:, :, None, None]).to(FP8), scales


def _tables(rng, lens, most, b):
    """Block tables of sequences of the given lengths in a pool of permuted blocks that has room
    for the longest ones (`most`) too."""
    need = (np.asarray(lens) + b - 1) // b
    blocks = math.ceil(1.05 * ((np.asarray(most) + b - 1) // b).sum()) + 2
    table = np.zeros((len(lens), max(1, need.max())), dtype=np.int32)
    table[np.arange(table.shape[1]) < need[:, None]] = rng.permutation(blocks)[:need.sum()]
    return torch.tensor(table, device="cuda"), blocks


def _ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _ragged(case):
    """New tokens (rows) of each sequence: all but the first a little fewer than the case says."""
    return [case["new"] - (37 * i) % max(1, case["new"] // 4) for i in range(case["seqs"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, hq, hkv, d, count = (case[k] for k in ("b", "hq", "hkv", "d", "seqs"))
    dt = DTYPES[case["dtype"]]
    new = [1] * count if case["op"] == "decode" else _ragged(case)
    if case["op"] == "append":
        old = [int(x) for x in rng.integers(0, case["old"] + 1, count)]
        lens = [o + n for o, n in zip(old, new)]
    elif case["op"] == "chunk":
        lens = [int(x) for x in rng.integers(max(case["new"], case["ctx"] * 7 // 8), case["ctx"] + 1, count)]
    elif case["op"] == "cross":       # an encoder may have said nothing at all
        lens = [int(x) for x in rng.integers(case["ctx"] // 4, case["ctx"] + 1, count)]
    else:
        low = 1 if case["spread"] else max(1, case["ctx"] * 15 // 16)
        lens = [int(x) for x in rng.integers(low, case["ctx"] + 1, count)]
    most = [case["old"] + n for n in new] if case["op"] == "append" else [max(case["ctx"], n) for n in new]
    table, blocks = _tables(rng, lens, most, b)
    seq = np.repeat(np.arange(count), new)
    tok = np.concatenate([np.arange(n) for n in new])
    st = dict(case=case, table=table, lens=_ints(lens), start=_ints(np.concatenate([[0], np.cumsum(new)])),
              max_len=max(lens), max_new=max(new), scale=d ** -0.5, seq=_ints(seq, torch.int64),
              tok=_ints(tok, torch.int64),
              pos=_ints(np.asarray(lens)[seq] - np.asarray(new)[seq] + tok, torch.int64))
    rows = len(seq)
    if case["op"] == "append":
        # the rows of one projection: q, k and v of a token lie beside each other
        qkv = torch.empty((rows, (hq + 2 * hkv), d), device="cuda").normal_(0.0, 1.0, generator=g)
        qkv *= torch.exp2(torch.empty((rows, 1, 1), device="cuda").normal_(0.0, 0.5, generator=g))
        qkv = qkv.to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["freq"] = 10000.0 ** (-2.0 * np.arange(case["rot"] // 2, dtype=np.float64) / max(1, case["rot"]))
        st["freq_gpu"] = torch.tensor(st["freq"], device="cuda")
    else:
        # scores of a few units, as trained attention has them
        st["q"] = torch.empty((rows, hq, d), device="cuda", dtype=dt).normal_(0.0, 3.0, generator=g)
    kind = case.get("kind", "block")
    if kind == "half":
        shape = (blocks, hkv, b, d)
        st["k_cache"] = torch.empty(shape, device="cuda", dtype=dt).normal_(0.0, 1.0, generator=g)
        st["v_cache"] = torch.empty(shape, device="cuda", dtype=dt).normal_(0.0, 1.0, generator=g)
    elif kind == "head":
        for name in ("k", "v"):
            st[name + "_scales"] = _ints(rng.uniform(0.008, 0.02, hkv), torch.float32)
            x = torch.empty((blocks, hkv, b, d), device="cuda").normal_(0.0, 1.0, generator=g)
            st[name + "_cache"] = (x / st[name + "_scales"][:, None, None]).clamp_(-448, 448).to(FP8)
    else:
        st["k_cache"], st["k_scales"] = _block_pool(g, blocks, case, 0.8)
        st["v_cache"], st["v_scales"] = _block_pool(g, blocks, case, 0.8)
    return st


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


def _append_rows(s, x, cache, scales):
    """Writes the rows x [T, Hkv, D] (fp32) into the cache in place."""
    case, hkv, b = s["case"], s["case"]["hkv"], s["case"]["b"]
    seq, pos = s["seq"], s["pos"]
    first = (s["lens"].long() - (s["start"][1:] - s["start"][:-1]).long())[seq]     # of the sequence's new tokens
    # touched blocks: (sequence, logical block) pairs, numbered along the tokens
    opens = (s["tok"] == 0) | (pos % b == 0)
    group = torch.cumsum(opens, 0) - 1
    at = torch.nonzero(opens)[:, 0]
    block = s["table"][seq[at], pos[at] // b].long()
    old_rows = (first[at] - pos[at] // b * b).clamp(min=0)                         # earlier tokens of the block
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)                   # [T, Hkv]
    most = torch.zeros((at.numel(), hkv), device="cuda").scatter_reduce(
        0, group[:, None].expand(-1, hkv), amax, "amax", include_self=True)
    before = scales[block, :hkv]
    after = _scale_for(most)
    after = torch.where(old_rows[:, None] > 0, torch.maximum(after, before), after)
    # earlier tokens in the new scale
    raw = cache.view(torch.uint8)
    codes = raw[block].view(FP8)
    told = (codes.float() * (before / after)[:, :, None, None]).to(FP8).view(torch.uint8)
    earlier = torch.arange(b, device="cuda")[None, :] < old_rows[:, None]
    raw[block] = torch.where(earlier[:, None, :, None], told, codes.view(torch.uint8))
    scales[block, :hkv] = after
    # the new tokens
    new = (x / after[group][:, :, None]).clamp(-448, 448).to(FP8).view(torch.uint8)
    raw[block[group], :, pos % b] = new


def _plain_append(s):
    case = s["case"]
    q, k = s["q"], s["k"].float()
    if case["rot"]:
        angle = s["pos"].double()[:, None, None] * s["freq_gpu"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q = _rotate(q, cos, sin, case["rot"], case["inter"]).to(q.dtype)
        k = _rotate(k, cos, sin, case["rot"], case["inter"])
    _append_rows(s, k, s["k_cache"], s["k_scales"])
    _append_rows(s, s["v"].float(), s["v_cache"], s["v_scales"])
    return _written(s, q)


def _written(s, q):
    out = {name: s[name] for name in ("k_cache", "v_cache", "k_scales", "v_scales")}
    return dict(out, q=q) if s["case"]["rot"] else out


def _gather(s, name):
    """[S, Hkv, W * B, D] in 32 bits."""
    case, cache, table = s["case"], s[name + "_cache"], s["table"].long()
    kind = case.get("kind", "block")
    if kind == "half":
        x = cache[table].float()
    else:
        scales = s[name + "_scales"]
        scales = scales[table, :case["hkv"]][..., None, None] if kind == "block" else scales[:, None, None]
        x = cache.view(torch.uint8)[table].view(FP8).float() * scales
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(s):
    case = s["case"]
    group = case["hq"] // case["hkv"]
    k, v = _gather(s, "k"), _gather(s, "v")
    t = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"].long()
    count, n = lens.numel(), s["max_new"]
    q = torch.zeros((count, n, case["hq"], case["d"]), device="cuda")
    q[s["seq"], s["tok"]] = s["q"].float()
    pos = (lens - 1)[:, None].expand(count, n).clone()
    if case["op"] == "chunk":
        pos[s["seq"], s["tok"]] = s["pos"]
    # rows [S, Hkv, n * G]: q . k for every row and token
    rows = q.unflatten(2, (case["hkv"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(rows * s["scale"], k.transpose(2, 3)).unflatten(2, (n, group))
    seen = (t <= pos[:, :, None])[:, None, :, None, :]
    x = x.masked_fill(~seen, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)            # a row that sees nothing is 0
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[s["seq"], s["tok"]].to(s["q"].dtype)


# --------------------------------------------------------------------------- the library

def _own_append(s):
    import paged_kv_cache_119_gb300 as pa
    case = s["case"]
    pools = (s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["lens"],
             s["start"])
    if not case["rot"]:
        pa.pa_append_fp8_block(*pools, max_query_len=s["max_new"])
        return _written(s, None)
    q = torch.empty((s["q"].shape[0], case["hq"], case["d"]), device="cuda", dtype=s["q"].dtype)
    pa.pa_rotary_and_append_fp8_block(q, s["q"], *pools, s["freq"], interleaved=case["inter"],
                                      max_query_len=s["max_new"])
    return _written(s, q)


def _own_attention(s):
    import paged_kv_cache_119_gb300 as pa
    case = s["case"]
    out = torch.empty_like(s["q"])
    kind = case.get("kind", "block")
    pools = (out, s["q"], s["k_cache"], s["v_cache"])
    if kind != "half":
        pools += (s["k_scales"], s["v_scales"])
    pools += (s["table"], s["lens"])
    shape = (s["scale"], case["hkv"], case["b"])
    if case["op"] == "decode":
        return pa.pa_decode_fp8_block(*pools, *shape, max_context_len=s["max_len"])
    call = {"chunk": pa.pa_chunk_attention_fp8_block} if case["op"] == "chunk" else {
        "half": pa.pa_cross_attention, "head": pa.pa_cross_attention_fp8, "block": pa.pa_cross_attention_fp8_block}
    return call[kind if case["op"] == "cross" else "chunk"](
        *pools, s["start"], *shape, max_query_len=s["max_new"], max_context_len=s["max_len"])


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attention(state) if own else _plain_attention(state)


# --------------------------------------------------------------------------- work

def work(case):
    hq, hkv, d, b, count = (case[k] for k in ("hq", "hkv", "d", "b", "seqs"))
    rows = count if case["op"] == "decode" else sum(_ragged(case))
    if case["op"] == "append":
        # q in and out where it turns, k and v in, their codes out, a scale in or out per block
        blocks = count + rows // b
        return {"bytes": rows * d * (2 * hkv * 3 + (4 * hq if case["rot"] else 0)) + 8 * blocks * hkv,
                "flops": rows * (3 * (hq + hkv) * case["rot"] + 4 * hkv * d)}
    size = 4 if case.get("kind", "block") == "half" else 2        # bytes of K and V of a token, head and dim
    per_token = hkv * (d * size + (8.0 / b if case.get("kind", "block") == "block" else 0))
    if case["op"] == "decode":
        length = (case["ctx"] + 1) / 2 if case["spread"] else case["ctx"] * 31 / 32
    else:
        length = case["ctx"] * (15 / 16 if case["op"] == "chunk" else 5 / 8)
    length = max(1.0, length)
    pairs = rows * (length - (rows / count / 2 if case["op"] == "chunk" else 0))
    return {"bytes": count * length * per_token + 4 * rows * hq * d, "flops": 4.0 * d * hq * max(pairs, rows)}


# --------------------------------------------------------------------------- in 64 bits

def _exact_scale(amax):
    s = 2.0 ** max(LOW, min(HIGH, math.ceil(math.log2(amax / 448.0)))) if amax > 0 else 2.0 ** LOW
    return s * 2.0 if amax > 448.0 * s and s < 2.0 ** HIGH else s


def exact(case, seed):
    s = prepare(case, seed)

    def append():
        out = {}
        angle = torch.outer(s["pos"].double(), s["freq_gpu"])
        turn = torch.polar(torch.ones_like(angle), angle)
        half = case["rot"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
        second = first + (1 if case["inter"] else half)
        turned = {"v": s["v"].double()}
        for name in ("q", "k"):
            y = s[name].double()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
            y[..., first], y[..., second] = z.real, z.imag
            turned[name] = y
        lens, start, table = s["lens"].tolist(), s["start"].tolist(), s["table"].tolist()
        b = case["b"]
        for name in ("k", "v"):
            pool = s[name + "_cache"].double()
            scales = s[name + "_scales"].double()
            old = scales.clone().cpu()
            for i, length in enumerate(lens):
                n = start[i + 1] - start[i]
                for at in range((length - n) // b, (length + b - 1) // b):
                    lo, hi = max(at * b, length - n), min((at + 1) * b, length)
                    block, x = table[i][at], turned[name][start[i] + lo - (length - n):start[i] + hi - (length - n)]
                    amax = x.abs().amax((0, 2)).tolist()
                    now = [_exact_scale(a) for a in amax]
                    if lo > at * b:
                        now = [max(a, o) for a, o in zip(now, old[block].tolist())]
                    now = torch.tensor(now, device="cuda", dtype=torch.float64)
                    if lo > at * b:
                        pool[block, :, :lo - at * b] *= (scales[block, :case["hkv"]] / now)[:, None, None]
                    pool[block, :, lo - at * b:hi - at * b] = (x / now[:, None]).transpose(0, 1)
                    scales[block, :case["hkv"]] = now
            out[name + "_cache"], out[name + "_scales"] = pool, scales
        written = {name: out[name] for name in ("k_cache", "v_cache", "k_scales", "v_scales")}
        return dict(written, q=turned["q"]) if case["rot"] else written

    if case["op"] == "append":
        return append()
    b, hkv, d = case["b"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    start = s["start"].tolist()
    kind = case.get("kind", "block")
    result = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        ids = s["table"][i, :(length + b - 1) // b].long()
        kv = []
        for name in ("k", "v"):
            pool = s[name + "_cache"]
            x = pool[ids].double() if kind == "half" else pool.view(torch.uint8)[ids].view(FP8).double()
            if kind == "block":
                x = x * s[name + "_scales"][ids, :hkv].double()[:, :, None, None]
            elif kind == "head":
                x = x * s[name + "_scales"].double()[:, None, None]
            kv.append(x.transpose(0, 1).reshape(hkv, -1, d)[:, :length])
        q = s["q"][start[i]:start[i + 1]].double()
        n = q.shape[0]
        hidden = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if case["op"] == "chunk":
            at = torch.arange(length - n, length, device="cuda")[:, None]
            hidden = torch.arange(length, device="cuda")[None, :] > at
        for h in range(hkv):
            x = torch.einsum("ngd,td->ngt", q[:, h * group:(h + 1) * group], kv[0][h]) * s["scale"]
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            result[start[i]:start[i + 1], h * group:(h + 1) * group] = torch.einsum(
                "ngt,td->ngd", torch.softmax(x, dim=-1), kv[1][h])
    return result
