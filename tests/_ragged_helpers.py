"""Plain forms of the ragged serving step's operators, and small inputs for them."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import _draft_helpers as H

BS, D = H.BS, H.D
NAN_CODE = 0x7F


# ---- attention to a window and the first tokens -------------------------------------

def seen_blocks(ctx, n, act, window, sinks):
    """Blocks that a token of a sequence sees."""
    w = act if window is None else window
    first = max(0, ctx - w + 1)
    return sorted(set(range(-(-min(sinks, first) // BS))) | set(range(first // BS, -(-act // BS)))) if n else []


def window_case(seed, ctx, new, NQ, NKV, layout, window, sinks, rows_behind=0, room=0, device="cpu"):
    """Inputs of one window_attention call. Blocks that no token sees have ids that
    are none, and cache bytes that no token sees are NaN codes."""
    rng = np.random.default_rng(seed)
    B = len(ctx)
    act = [c + n for c, n in zip(ctx, new)]
    need = [seen_blocks(c, n, a, window, sinks) for c, n, a in zip(ctx, new, act)]
    NB = sum(map(len, need)) + 2
    ids = rng.permutation(NB)
    bt = np.where(rng.random((B, max([-(-a // BS) for a in act] + [1]) + room)) < 0.5, -1, 10 ** 6).astype(np.int32)
    at = 0
    for b in range(B):
        bt[b, need[b]] = ids[at:at + len(need[b])]
        at += len(need[b])
    T = sum(new) + rows_behind
    sh = H.cache_shape(layout, NB, NKV)
    c = dict(B=B, NQ=NQ, NKV=NKV, layout=layout, window=window, sinks=sinks, most=max(list(new) + [1]),
             act=torch.tensor(act, dtype=torch.int32), bt=torch.from_numpy(bt),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)),
             kc=H.codes(rng, sh + (D,)), vc=H.codes(rng, sh + (D,)),
             ks=torch.from_numpy(rng.uniform(0.005, 0.012, sh).astype(np.float32)),
             q=H.codes(rng, (T, NQ, D)),
             qs=torch.from_numpy(rng.uniform(0.005, 0.012, (T, NQ)).astype(np.float32)),
             vs=torch.from_numpy(rng.uniform(0.005, 0.012, (B, NKV, D)).astype(np.float32)))
    # what no token sees
    seen = torch.zeros((NB, BS), dtype=torch.bool)
    for b in range(B):
        pos = torch.arange(act[b])
        first = max(0, ctx[b] - (act[b] if window is None else window) + 1)
        pos = pos[(pos >= first) | (pos < sinks)] if new[b] else pos[:0]
        seen[torch.from_numpy(bt[b]).long()[pos // BS], pos % BS] = True
    for k in ("kc", "vc", "ks"):
        H.by_position(c[k], layout)[~seen] = NAN_CODE if k != "ks" else math.nan
    return {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def window_reference(c, scale=None):
    """(out, bound) in 64 bits, [T, NQ, D]; NaN rows behind the last sequence. The
    bound counts the roundings as tree_reference's does: the output's to BF16 (2^-8 of
    the value), P's to FP16 (2^-11 each), an FP32 score's error (128 products and two
    scales, 2^-24 each, on the sum of magnitudes), twice since it enters the numerator
    and the sum, the exponential (2^-20), and the weights too small for FP16 (2^-31 of
    the largest, each)."""
    NQ, NKV, dev = c["NQ"], c["NKV"], c["q"].device
    G = NQ // NKV
    scale = D ** -0.5 if scale is None else scale
    T = c["q"].shape[0]
    out = torch.full((T, NQ, D), math.nan, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    kc, vc, ks = (H.by_position(c[k], c["layout"]) for k in ("kc", "vc", "ks"))
    val = lambda x: x.view(H.F8).double()  # noqa: E731
    for b in range(c["B"]):
        act = max(0, min(int(c["act"][b]), c["bt"].shape[1] * BS))
        t0, t1 = (max(0, min(int(c["cu"][b + i]), T)) for i in (0, 1))
        out[t0:t1] = 0
        live = min(t1, t0 + c.get("max_tokens", T))
        w = act if c["window"] is None else c["window"]
        for r0 in range(t0, live, 512):
            r1 = min(live, r0 + 512)
            p = torch.arange(r0, r1, device=dev) - t1 + act
            lo = max(0, int(p[0]) - w + 1)
            pos = torch.arange(max(0, int(p[-1]) + 1), device=dev)
            pos = pos[(pos >= lo) | (pos < c["sinks"])]
            if len(pos) == 0:
                continue
            far = p[:, None] - pos[None]
            see = (far >= 0) & ((far < w) | (pos < c["sinks"])[None])
            blk = c["bt"][b].long()[pos // BS]
            blk = torch.where((blk < 0) | (blk >= kc.shape[0]), 0, blk)
            for h in range(NKV):
                hs = slice(h * G, (h + 1) * G)
                K = val(kc[blk, pos % BS, h]) * ks[blk, pos % BS, h].double()[:, None]
                V = val(vc[blk, pos % BS, h])
                q = val(c["q"][r0:r1, hs]) * c["qs"][r0:r1, hs, None].double()
                s = torch.einsum("ngd,kd->ngk", q, K) * scale
                mag = torch.einsum("ngd,kd->ngk", q.abs(), K.abs()) * abs(scale)
                s = torch.where(see[:, None], s, -math.inf)
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
                L = e.sum(-1, keepdim=True)
                one = torch.where(L == 0, 1.0, L)
                vsc = c["vs"][b, h].double()
                o = torch.einsum("ngk,kd->ngd", e, V) / one * vsc
                mass = torch.einsum("ngk,kd->ngd", e, V.abs()) / one * vsc
                err = torch.where(see[:, None], mag, 0).amax(-1, keepdim=True) * 130 * 2.0 ** -24
                vmax = V.abs().amax() * vsc
                out[r0:r1, hs] = o
                tol[r0:r1, hs] = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -20 + 2 * err) * mass \
                    + len(pos) * 2.0 ** -31 * vmax + 2.0 ** -30
    return out, tol


# ---- the plan ------------------------------------------------------------------------

def plan_reference(act, new, pool, head, bt, T, NB, bs):
    """(block table, slots, positions, token_batch, cu, new lengths, new head)."""
    bt = np.array(bt)
    B, W = bt.shape
    slots, pos, batch = np.full(T, -1, np.int64), np.zeros(T, np.int64), np.zeros(T, np.int64)
    head = min(max(head, 0), len(pool))
    rows = taken = granted = 0
    cu, out_act = [0], []
    for b in range(B):
        a, n = max(int(act[b]), 0), max(int(new[b]), 0)
        first = min(rows, T)
        rows += n
        ok = a + n <= W * bs and rows <= T
        have = -(-a // bs)
        need = -(-(a + n) // bs) - have if ok else 0
        taken += need
        if need and head + taken > len(pool):
            ok = False
        if ok and need:
            bt[b, have:have + need] = pool[head + taken - need:head + taken]
            granted = taken
        for i in range(first, min(rows, T)):
            p = a + i - first
            pos[i], batch[i] = min(p, 2 ** 31 - 1), b
            if ok and 0 <= bt[b, p // bs] < NB:
                slots[i] = int(bt[b, p // bs]) * bs + p % bs
        cu.append(min(rows, T))
        out_act.append(a + n if ok else a)
    return bt, slots, pos, batch, np.array(cu), np.array(out_act, np.int64), np.array([head + granted])


# ---- log probabilities ---------------------------------------------------------------

def logprob_reference(x, tok, k):
    """(logprobs, ranks, entropy, top ids, top logprobs) in 64 bits of rows without NaN
    and +inf."""
    x = x.double()
    R, V = x.shape
    m = x.amax(-1, keepdim=True)
    none = m == -math.inf
    e = torch.exp(x - torch.where(none, 0.0, m))
    L = e.sum(-1, keepdim=True)
    logz = torch.where(none, 0.0, m + torch.log(L))
    lp = x - logz
    ent = -torch.where(e > 0, e / torch.where(none, 1.0, L) * lp, 0.0).sum(-1)
    inside = (tok >= 0) & (tok < V)
    at = torch.where(inside, tok, 0).long()[:, None]
    own = torch.gather(x, 1, at)
    rank = torch.where(inside, (x > own).sum(-1), -1)
    order = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :k]
    return torch.where(inside, torch.gather(lp, 1, at)[:, 0], math.nan), rank, ent, order, torch.gather(lp, 1, order)
