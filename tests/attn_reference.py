"""Paged inputs and a plain 64-bit reference for the modified-score and shared-prefix calls.

A case holds each sequence's dense K and V in 64 bits (the values the pool stands for).  In
the pools every slot of a token that no row sees is NaN, and table entries of blocks without
a seen token are -1, so a read outside the seen tokens shows.

Tolerance of an attention output, derived: the fp32 dot of D <= 128 products of rows with
sum |q_i k_i| scale <= 16 is within 128 * 2^-24 * 16 = 1.2e-4 of the exact score (the cap,
2^-20 relative, and the distance term, 2^-24 of it, add less than 1e-5 where a token still
has weight); weights are then within e^(2 * 1.3e-4), so the output within
2 * 1.3e-4 * max |v - o| <= 5.2e-4 max |v|.  The tcgen05 chunk kernel rounds each
probability once to f16: 2^-11 max |v| more.  A native output is rounded once: eps / 2.
"""
import numpy as np
import torch

ROWS_TOL = 5.2e-4
CHUNK_TOL = ROWS_TOL + 2.0 ** -11
FP8 = torch.float8_e4m3fn


class Case:
    pass


def visible(L, n, window, glob):
    """[n, L] bool: which tokens the last n rows of a sequence of L tokens see."""
    pos = np.arange(L - n, L)[:, None]
    t = np.arange(L)[None, :]
    v = t <= pos
    if window:
        v &= pos - t < window
    return v | (t < glob)


def build(seed, lens, new, Hq, Hkv, D, B, dtype, fp8=False, window=0, glob=None, shared=None,
          kstd=1.0, extra_blocks=3):
    """shared: list of (first sequence, last + 1, tokens) groups whose blocks are the same."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = Case()
    S = len(lens)
    c.lens, c.new, c.Hq, c.Hkv, c.D, c.B, c.fp8, c.dtype = lens, new, Hq, Hkv, D, B, fp8, dtype
    c.window, c.glob = window, glob
    need = [(L + B - 1) // B for L in lens]
    N = sum(need) + extra_blocks
    ids = rng.permutation(N)
    W = max(1, max(need)) + 1
    table = np.full((S, W), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    c.shared_len = np.zeros(S, dtype=np.int32)
    for a, b, P in shared or []:
        for s in range(a, b):
            table[s, :P // B] = table[a, :P // B]
            c.shared_len[s] = P
    scale = [(torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.004) for _ in range(2)]
    pools, dense = [], []
    for i, std in enumerate((kstd, 1.0)):
        x = torch.randn((N, Hkv, B, D), generator=g, device="cuda") * std
        if fp8:
            codes = (x / scale[i][:, None, None]).clamp(-448, 448).to(FP8)
            value = codes.float().double() * scale[i].double()[:, None, None]
            pools.append(codes.view(torch.uint8).clone())
        else:
            value = x.to(dtype).double()
            pools.append(x.to(dtype))
        dense.append(value)
    tt = torch.tensor(table, device="cuda").long()
    c.K = [dense[0][tt[s, :need[s]]].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[s]] for s in range(S)]
    c.V = [dense[1][tt[s, :need[s]]].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[s]] for s in range(S)]
    c.seen = []
    live = np.zeros((N, B), bool)
    for s in range(S):
        v = visible(lens[s], new[s], window, min(glob[s], lens[s]) if glob is not None else 0) \
            if lens[s] and new[s] else np.zeros((max(new[s], 1), lens[s]), bool)
        c.seen.append(v)
        any_row = v.any(0)
        for t in np.flatnonzero(any_row):
            live[table[s, t // B], t % B] = True
        for j in range(need[s]):
            if not any_row[j * B:(j + 1) * B].any() and not c.shared_len[s]:
                table[s, j] = -1
    dead = torch.tensor(~live, device="cuda")[:, None, :, None].expand(N, Hkv, B, D)
    for x in pools:
        x.masked_fill_(dead, 0x7f if fp8 else float("nan"))
    c.k_cache, c.v_cache = [x.view(FP8) if fp8 else x for x in pools]
    c.k_scale, c.v_scale = scale
    c.table = torch.tensor(table, device="cuda")
    c.context_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    start = np.concatenate([[0], np.cumsum(new)])
    c.query_start = torch.tensor(start, dtype=torch.int32, device="cuda")
    R = int(start[-1])
    c.q = torch.randn((R, Hq, D), generator=g, device="cuda").to(dtype)
    c.global_lens = None if glob is None else torch.tensor(glob, dtype=torch.int32, device="cuda")
    c.scale = D ** -0.5
    c.pools = (c.k_cache, c.v_cache) + ((c.k_scale, c.v_scale) if fp8 else ())
    return c


def reference(c, softcap=0.0, slopes=None, scale=None):
    """[R, Hq, D] in 64 bits (numpy) and max |v|; a row that sees nothing is 0."""
    scale = c.scale if scale is None else scale
    G = c.Hq // c.Hkv
    out, r = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda"), 0
    for s, (L, n) in enumerate(zip(c.lens, c.new)):
        if L and n:
            q = c.q[r:r + n].double().view(n, c.Hkv, G, c.D)
            x = torch.einsum("nhgd,htd->hngt", q, c.K[s]) * scale
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                pos = torch.arange(L - n, L, device="cuda")[:, None]
                dist = (pos - torch.arange(L, device="cuda")[None, :]).abs().double()
                x = x - slopes.double().view(c.Hkv, 1, G, 1) * dist[None, :, None, :]
            seen = torch.tensor(c.seen[s], device="cuda")
            x = x.masked_fill(~seen[None, :, None, :], float("-inf"))
            p = torch.softmax(x, -1)
            out[r:r + n] = torch.einsum("hngt,htd->nhgd", p, c.V[s]).reshape(n, c.Hq, c.D)
        r += n
    vmax = max((v.abs().max().item() for v in c.V if v.numel()), default=1.0)
    return out.cpu().numpy(), vmax


def check(got, ref, vmax, tol):
    """got against ref: tol * vmax, plus half a step of a 16-bit output."""
    err = np.abs(got.double().cpu().numpy() - ref)
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    limit = tol * vmax + half * (np.abs(ref) + tol * vmax)
    assert np.isfinite(err).all(), "an output is not finite"
    assert (err <= limit).all(), f"off by {float((err - limit).max()):.3e} beyond the tolerance"
