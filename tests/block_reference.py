"""Block-scaled E4M3 inputs and plain references: the append in the order of its definition, and
attention (causal chunk, decode, cross) in 64 bits.

In the pools every slot of a token that no row sees is NaN (code 0x7f), the scales of unused blocks
are NaN, and table entries past a sequence's last block are -1.
"""
import numpy as np
import torch

FP8 = torch.float8_e4m3fn
LOW, HIGH = -48, 48


def decode(codes):
    """Values of uint8 codes in 64 bits (CPU)."""
    table = torch.arange(256, dtype=torch.uint8).view(FP8).double()
    return table[codes.cpu().long()]


def encode(x):
    """uint8 codes of fp32 values (CPU): nearest, ties to even, saturating, NaN stays NaN."""
    return x.float().cpu().clamp(-448, 448).to(FP8).view(torch.uint8)


def same(a, b):
    """Equal codes (all NaN codes are one) or scales."""
    if a.dtype == torch.uint8:
        a, b = [torch.where(x & 0x7f == 0x7f, torch.tensor(0x7f, dtype=torch.uint8), x) for x in (a, b)]
    return torch.equal(a, b)


def scale_for(amax):
    """The smallest power of two s in range with amax <= 448 s."""
    s = 2.0 ** LOW
    while s < 2.0 ** HIGH and amax > 448.0 * s:
        s *= 2.0
    return s


def rotate(x, positions, freq, interleaved, magnitude=1.0):
    """[T, H, D] turned by its positions, in 64 bits (CPU)."""
    y = x.double().cpu().clone()
    half = len(freq)
    if not half:
        return y
    a = torch.arange(half) * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    angle = torch.outer(positions.double().cpu(), torch.tensor(freq, dtype=torch.float64))
    c, s = magnitude * torch.cos(angle)[:, None, :], magnitude * torch.sin(angle)[:, None, :]
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def append(x, codes, scales, table, lens, new, B):
    """The definition: rows x [T, Hkv, D] (fp32 or exact in it) appended to codes (uint8 CPU
    [N, Hkv, B, D]) and scales (fp32 CPU [N, stride]) in place."""
    row = 0
    Hkv = codes.shape[1]
    for s, (L, n) in enumerate(zip(lens, new)):
        at = L - n
        while at < L:
            lb = at // B
            end = min(L, lb * B + B)
            block, r0, cnt = int(table[s, lb]), at - lb * B, end - at
            rows = x[row:row + cnt]
            row += cnt
            at = end
            if block < 0 or block >= codes.shape[0]:
                continue
            for h in range(Hkv):
                v = rows[:, h].float()
                fin = v[torch.isfinite(v)].abs()
                sc = scale_for(float(fin.max()) if fin.numel() else 0.0)
                if r0:
                    old = min(max(float(scales[block, h]), 2.0 ** LOW), 2.0 ** HIGH)
                    if sc > old:
                        ratio = np.float32(old) / np.float32(sc)
                        codes[block, h, :r0] = encode(decode(codes[block, h, :r0]).float() * float(ratio))
                    sc = max(sc, old)
                scales[block, h] = sc
                codes[block, h, r0:r0 + cnt] = encode(v / np.float32(sc))


class Case:
    pass


def build(seed, lens, new, Hq, Hkv, D, B, dtype, causal=True, vscale=(-8, -5), pow2=True, pad=True, kind="block",
          kstd=1.0):
    """kind: "block", "head" (one scale per kv head) or "half" (caches of the queries' type)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    c = Case()
    c.lens, c.new, c.Hq, c.Hkv, c.D, c.B, c.dtype, c.causal = lens, new, Hq, Hkv, D, B, dtype, causal
    need = [(L + B - 1) // B for L in lens]
    N = sum(need) + 3
    ids = rng.permutation(N)
    c.table_np = np.full((len(lens), max(1, max(need)) + 1), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        c.table_np[s, :n] = ids[at:at + n]
        at += n
    stride = (Hkv + 3) // 4 * 4 if pad else Hkv
    live = torch.zeros((N, B), dtype=torch.bool)
    for s, L in enumerate(lens):
        for t in range(L):
            live[c.table_np[s, t // B], t % B] = True
    dead = ~live[:, None, :, None].expand(N, Hkv, B, D)
    unused = ~live.any(1)
    dense, c.pools, c.scales = [], [], []
    for which, std in enumerate((kstd, 1.0)):
        x = torch.randn((N, Hkv, B, D), generator=g)
        if kind == "half":
            pool = (x * std).to(dtype)
            dense.append(pool.double())
            pool[dead] = float("nan")
            c.pools.append(pool.cuda())
            continue
        if kind == "head":
            sc = (torch.rand(Hkv, generator=g) * 0.01 + 0.004)
            full = sc[None, :].expand(N, Hkv)
            x = x * std
        else:
            lo, hi = (-8, -5) if which == 0 else vscale
            e = torch.tensor(rng.uniform(lo, hi, (N, Hkv)))
            full = torch.exp2(e.round() if pow2 else e).float()
            # (values of each block in proportion to its V scale, K values of one size)
            x = x * std if which == 0 else x * full[:, :, None, None] * 100.0
        codes = encode(x / full[:, :, None, None])
        dense.append(decode(codes) * full.double()[:, :, None, None])
        codes[dead] = 0x7f
        c.pools.append(codes.cuda().view(FP8))
        if kind == "head":
            c.scales.append(sc.cuda())
        else:
            full = full.clone()
            full[unused] = float("nan")
            padded = torch.full((N, stride), float("nan"))
            padded[:, :Hkv] = full
            c.scales.append(padded.cuda())
            if which == 1:
                c.vfull = full
    tt = torch.tensor(c.table_np).long()
    c.K = [dense[0][tt[s, :need[s]]].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[s]] for s in range(len(lens))]
    c.V = [dense[1][tt[s, :need[s]]].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[s]] for s in range(len(lens))]
    c.table = torch.tensor(c.table_np).cuda()
    c.context_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    start = np.concatenate([[0], np.cumsum(new)])
    c.query_start = torch.tensor(start, dtype=torch.int32).cuda()
    c.q = torch.randn((int(start[-1]), Hq, D), generator=g).to(dtype).cuda()
    c.scale = D ** -0.5
    c.args = (*c.pools, *c.scales, c.table, c.context_lens)
    return c


def attend(c):
    """([R, Hq, D] in 64 bits, the same sums of |p v|): a row that sees nothing is 0."""
    G = c.Hq // c.Hkv
    out = np.zeros(tuple(c.q.shape))
    size = np.zeros(tuple(c.q.shape))
    q_all, r = c.q.double().cpu(), 0
    for s, (L, n) in enumerate(zip(c.lens, c.new)):
        if L and n:
            q = q_all[r:r + n].view(n, c.Hkv, G, c.D)
            x = torch.einsum("nhgd,htd->hngt", q, c.K[s]) * c.scale
            if c.causal:
                hidden = torch.arange(L)[None, :] > torch.arange(L - n, L)[:, None]
                x = x.masked_fill(hidden[None, :, None, :], float("-inf"))
            p = torch.softmax(x, -1)
            out[r:r + n] = torch.einsum("hngt,htd->nhgd", p, c.V[s]).reshape(n, c.Hq, c.D).numpy()
            size[r:r + n] = torch.einsum("hngt,htd->nhgd", p, c.V[s].abs()).reshape(n, c.Hq, c.D).numpy()
        r += n
    return out, size
