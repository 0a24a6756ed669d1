"""Plain 64-bit forms of the speculative decode step's operators, and small
inputs for them (random trees, paged caches of random codes)."""
from __future__ import annotations

import numpy as np
import torch

BS = 128
D = 128
F8 = torch.float8_e4m3fn


def codes(rng, shape, std=150.0):
    """E4M3 codes (no NaN) of normal values."""
    x = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * std).clamp(-448, 448)
    return x.to(F8).view(torch.uint8)


def value(c):
    return c.cpu().view(F8).double()


def cache_shape(layout, NB, NKV):
    return (NB, BS, NKV) if layout == 0 else (NB, NKV, BS)


def by_position(cache, layout):
    """A cache as [block, offset, head, ...]."""
    return cache if layout == 0 else cache.transpose(1, 2)


def random_tree(rng, n, width=4):
    return [-1] + [int(rng.integers(max(0, s - width), s)) for s in range(1, n)]


def ancestor_mask(parents):
    n = len(parents)
    m = np.zeros((n, n), bool)
    for s in range(n):
        if parents[s] >= 0:
            m[s] = m[parents[s]]
        m[s, s] = True
    return m


def tables(rng, need, width, spare=2):
    """Block tables of `need` blocks a sequence from one shuffled pool, -1 behind."""
    NB = int(sum(need)) + spare
    ids = rng.permutation(NB)
    bt = np.full((len(need), width), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        bt[b, :m] = ids[at:at + m]
        at += m
    return bt, NB


def tree_case(seed, ctx, S1, NQ, NKV, layout, n=None, width=None, room=0):
    """Inputs of one tree_decode call, on the CPU."""
    rng = np.random.default_rng(seed)
    B = len(ctx)
    n = np.full(B, S1, np.int32) if n is None else np.asarray(n, np.int32)
    act = (np.asarray(ctx) + n).astype(np.int32)
    need = [max(1, -(-int(a) // BS)) for a in act]
    bt, NB = tables(rng, need, (width or max(need)) + room)
    sh = cache_shape(layout, NB, NKV)
    c = dict(B=B, S1=S1, NQ=NQ, NKV=NKV, layout=layout, ctx=list(ctx), n=torch.from_numpy(n),
             act=torch.from_numpy(act), bt=torch.from_numpy(bt), kc=codes(rng, sh + (D,)),
             vc=codes(rng, sh + (D,)),
             ks=torch.from_numpy(rng.uniform(0.005, 0.012, sh).astype(np.float32)),
             q=codes(rng, (B * S1, NQ, D)),
             qs=torch.from_numpy(rng.uniform(0.005, 0.012, (B * S1, NQ)).astype(np.float32)),
             vs=torch.from_numpy(rng.uniform(0.005, 0.012, (B, NKV, D)).astype(np.float32)))
    mask = np.zeros((B, S1, S1), bool)
    for b in range(B):
        mask[b] = ancestor_mask(random_tree(rng, S1))
    c["mask"] = torch.from_numpy(mask)
    return c


def tree_reference(c, scale=None):
    """(out, bound) in 64 bits, [B*S1, NQ, D]. The bound counts the roundings:
    the output's to BF16 (2^-8 of the value), P's to FP16 (2^-11 each), an
    FP32 score's error (128 products and two scales, 2^-24 each, on the sum
    of magnitudes), twice since it enters the numerator and the sum, the
    exponential (2^-20), and the weights too small for FP16 (2^-31 of the
    largest, each). Where one key is left the quotient is that key's value."""
    B, S1, NQ, NKV = c["B"], c["S1"], c["NQ"], c["NKV"]
    G = NQ // NKV
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B * S1, NQ, D), dtype=torch.float64)
    tol = torch.zeros_like(out)
    kc, vc, ks = (by_position(c[k], c["layout"]) for k in ("kc", "vc", "ks"))
    for b in range(B):
        act = min(int(c["act"][b]), c["bt"].shape[1] * BS)
        n = max(0, min(int(c["n"][b]), S1, act))
        if act <= 0 or n == 0:
            continue
        pos = torch.arange(act)
        blk = c["bt"][b].long()[pos // BS]
        blk = torch.where((blk < 0) | (blk >= kc.shape[0]), 0, blk)
        see = torch.ones((n, act), dtype=torch.bool)
        see[:, act - n:] = c["mask"][b, :n, :n].bool()
        for h in range(NKV):
            K = value(kc[blk, pos % BS, h]) * ks[blk, pos % BS, h].double()[:, None]
            V = value(vc[blk, pos % BS, h])
            hs = slice(h * G, (h + 1) * G)
            q = value(c["q"][b * S1:b * S1 + n, hs]) * c["qs"][b * S1:b * S1 + n, hs, None].double()
            s = torch.einsum("ngd,kd->ngk", q, K) * scale
            mag = torch.einsum("ngd,kd->ngk", q.abs(), K.abs()) * abs(scale)
            s = torch.where(see[:, None], s, -np.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(m == -np.inf, 0.0, m))
            L = p.sum(-1, keepdim=True)
            one = torch.where(L == 0, 1.0, L)
            vsc = c["vs"][b, h].double()
            o = torch.einsum("ngk,kd->ngd", p, V) / one * vsc
            mass = torch.einsum("ngk,kd->ngd", p, V.abs()) / one * vsc
            err = torch.where(see[:, None], mag, 0).amax(-1, keepdim=True) * 130 * 2.0 ** -24
            vmax = V.abs().amax() * vsc
            out[b * S1:b * S1 + n, hs] = o
            tol[b * S1:b * S1 + n, hs] = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -20 + 2 * err) * mass \
                + act * 2.0 ** -31 * vmax + 2.0 ** -30
    return out, tol


FIX = 2.0 ** 45


def weights(r):
    r = np.nan_to_num(np.asarray(r, np.float64), nan=0.0)
    return np.floor(np.clip(r, 0.0, 1.0) * FIX).astype(np.int64)


def verify_reference(p, q, tok, par, u, n):
    """accepted, path, tokens from the definition; R and the products as it states them."""
    B, S1, V = p.shape
    accepted = np.zeros(B, np.int32)
    path = np.full((B, S1), -1, np.int32)
    tokens = np.full((B, S1), -1, np.int32)
    for b in range(B):
        if n[b] <= 0:
            continue
        cur, acc, R, z = 0, 1, p[b, 0].copy(), 1.0
        path[b, 0] = 0
        for s in range(1, min(int(n[b]), S1)):
            x = int(tok[b, s])
            if par[b, s] != cur or par[b, s] >= s or not 0 <= x < V:
                continue
            Q = float(q[b, cur, x]) if q is not None else 1.0
            if float(u[b, s]) * z * Q < float(R[x]):
                cur, R, z = s, p[b, s].copy(), 1.0
                path[b, acc] = s
                tokens[b, acc - 1] = x
                acc += 1
            elif q is not None:
                R = np.maximum(R - (np.float32(z) * q[b, cur]).astype(np.float32), np.float32(0))
                z = float(np.float32(float(weights(R).sum()) / FIX))
            else:
                z -= float(R[x])
                R[x] = 0
        W = weights(R)
        if W.sum() == 0:
            W = weights(p[b, cur])
        total = int(W.sum())
        if total:
            t = min(int(float(u[b, 0]) * float(total)), total - 1)
            tokens[b, acc - 1] = int(np.searchsorted(np.cumsum(W), t, side="right"))
        accepted[b] = acc
    return accepted, path, tokens


def norm_rope_reference(x, w, cos_sin, pos, inter, eps):
    """y in 64 bits, [T, H, D]."""
    x = x.double()
    y = x
    if w is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is not None and cos_sin.shape[1]:
        rd = cos_sin.shape[1]
        cs = cos_sin.double()[pos.long().clamp(0, cos_sin.shape[0] - 1)]
        i = torch.arange(rd // 2)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
        a, b, c, s = y[..., ia], y[..., ib], cs[:, None, :rd // 2], cs[:, None, rd // 2:]
        y = y.clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y
