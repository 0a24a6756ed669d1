"""What is measured of the operators of a ragged serving step (requests bring one
token or a prompt's chunk each): the cases, their plain forms in elementary torch
operations, and the library's calls.

  plan     plan_batch: block tables, slots and positions from request lengths
  append   qkv_norm_mrope_append: the append whose rotation takes each pair's angle
           from one of several position axes (time, height, width)
  window   window_attention: a sliding window and the first tokens, over the FP8 cache
  logp     token_logprobs: log probabilities, ranks, entropy and top alternatives
"""
import math
import random

import torch

own = False

D = 128
BS = 128
F8 = torch.float8_e4m3fn


def _pa():
    import fp8_paged_kv_block_gb300 as pa
    return pa


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 requests, one token each: latency
        dict(name="plan_decode", op="plan", B=64, chunks=0, lo=1, hi=8192, T=64, plan=1),
        # many requests, a quarter of them with a prompt's chunk, in a padded batch
        dict(name="plan_mixed", op="plan", B=1000, chunks=250, lo=0, hi=16384, T=65536, plan=2),
        # new tokens of 16 requests, contiguous sections of axes: latency
        dict(name="append_decode", op="append", T=16, NQ=96, NKV=8, rd=128, axes="sections", inter=False,
             dtype="bf16", layout="bsnd", B=16),
        # an odd batch in FP32, axes in turn, paired rotation of half a head
        dict(name="append_odd", op="append", T=777, NQ=48, NKV=8, rd=64, axes="turns", inter=True,
             dtype="f32", layout="bnbd", B=48),
        # the chunk of a prompt with images
        dict(name="append_images", op="append", T=8192, NQ=96, NKV=8, rd=128, axes="sections", inter=False,
             dtype="bf16", layout="bsnd", B=4),
        # one request's next token, a short window: latency
        dict(name="window_one", op="window", B=1, most=1, chunks=0, NQ=16, NKV=4, lo=700, hi=5000, window=512,
             sinks=4, plan=3, layout="bsnd"),
        # a decode batch of long requests, whose blocks behind the window are given back
        dict(name="window_decode", op="window", B=64, most=1, chunks=0, NQ=96, NKV=8, lo=2000, hi=60000,
             window=4096, sinks=64, plan=4, layout="bsnd"),
        # decoding requests and chunks of odd sizes in one batch
        dict(name="window_mixed", op="window", B=37, most=509, chunks=6, NQ=96, NKV=8, lo=1, hi=9000, window=1000,
             sinks=5, plan=5, layout="bnbd"),
        # two long prompts at once
        dict(name="window_prompt", op="window", B=2, most=5000, chunks=2, NQ=96, NKV=8, lo=0, hi=6000,
             window=4096, sinks=128, plan=6, layout="bsnd"),
        # the token just drawn, odd vocabulary: latency
        dict(name="logp_one", op="logp", R=1, V=32003, top=5, dtype="f32", pad=0),
        # a decode batch with twenty alternatives, BF16 logits
        dict(name="logp_batch", op="logp", R=250, V=131072, top=20, dtype="bf16", pad=0),
        # a prompt's tokens scored, padded rows, no alternatives
        dict(name="logp_prompt", op="logp", R=4096, V=50000, top=0, dtype="f32", pad=48),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "window", "window", "logp"])
    heads = rng.choice([(96, 8), (48, 8), (12, 2), (12, 1), (16, 4), (8, 8), (4, 1)])
    layout = rng.choice(["bsnd", "bnbd"])
    plan = rng.randrange(1, 1 << 30)
    if op == "plan":
        B = _log_int(rng, 1, 1000)
        chunks = rng.choice([0, B // 4])
        return dict(op=op, B=B, chunks=chunks, lo=rng.choice([0, 1]), hi=_log_int(rng, 100, 16384),
                    T=_log_int(rng, B, 4 * B) if chunks == 0 else _log_int(rng, 8 * B, 64 * B), plan=plan)
    if op == "append":
        return dict(op=op, T=_log_int(rng, 1, 8192), NQ=heads[0], NKV=heads[1], rd=rng.choice([32, 64, 128]),
                    axes=rng.choice(["sections", "turns"]), inter=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), layout=layout, B=_log_int(rng, 1, 64))
    if op == "window":
        window, sinks = _log_int(rng, 16, 4096), rng.choice([0, 1, 4, 64, 200])
        kind = rng.choice(["decode", "mixed", "prompt"])
        if kind == "decode":
            return dict(op=op, B=_log_int(rng, 1, 64), most=rng.choice([1, 1, 2, 4]), chunks=0, NQ=heads[0],
                        NKV=heads[1], lo=rng.choice([1, 1000]), hi=_log_int(rng, 1000, 60000), window=window,
                        sinks=sinks, plan=plan, layout=layout)
        if kind == "mixed":
            B = _log_int(rng, 2, 40)
            return dict(op=op, B=B, most=_log_int(rng, 5, 500), chunks=(B + 3) // 4, NQ=heads[0], NKV=heads[1], lo=1,
                        hi=_log_int(rng, 500, 9000), window=window, sinks=sinks, plan=plan, layout=layout)
        B = rng.choice([1, 2])
        return dict(op=op, B=B, most=_log_int(rng, 500, 5000), chunks=B, NQ=heads[0], NKV=heads[1], lo=0,
                    hi=_log_int(rng, 2, 6000), window=window, sinks=sinks, plan=plan, layout=layout)
    V = _log_int(rng, 1000, 131072)
    return dict(op=op, R=_log_int(rng, 1, min(4096, 130_000_000 // V)), V=V, top=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["f32", "bf16"]), pad=rng.choice([0, 0, 5, 64]))


def _requests(case):
    """Positions in the cache before the step and new tokens of each request, from
    the case alone: `chunks` requests, spread over the batch, bring prompt chunks."""
    r = random.Random(case["plan"])
    B, chunks = case["B"], case["chunks"]
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    if case["op"] == "plan":
        # chunks that fill about the batch's rows
        room = max(1, (case["T"] - B) // max(1, chunks))
        new = [1] * B
        for b in r.sample(range(B), chunks):
            new[b] = r.randint(1, room)
    else:
        new = [case["most"] if chunks == 0 else 1] * B
        for b in r.sample(range(B), chunks):
            new[b] = r.randint((case["most"] + 1) // 2, case["most"])
    return ctx, new


def _pairs(case):
    """(query, key) pairs a head, and the distinct positions of the cache that count."""
    ctx, new = _requests(case)
    w, s = case["window"], case["sinks"]
    pairs = keys = 0
    for c, n in zip(ctx, new):
        first = max(0, c - w + 1)
        keys += c + n - first + min(s, first)
        # sum over the tokens of min(p + 1, w) and of the sinks before the window
        p0, p1 = c, c + n - 1
        full = max(0, p1 - max(p0, w - 1) + 1)
        pairs += full * w + sum(p + 1 for p in range(p0, min(p1 + 1, w - 1)))
        pairs += sum(min(s, p - w + 1) for p in range(max(p0, w), p1 + 1))
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _requests(case)
        blocks = sum((c + n + BS - 1) // BS - (c + BS - 1) // BS for c, n in zip(ctx, new))
        return dict(bytes=case["T"] * 12 + case["B"] * 20 + blocks * 8, flops=0)
    if op == "append":
        rows = case["T"] * (case["NQ"] + 2 * case["NKV"])
        size = 2 if case["dtype"] == "bf16" else 4
        b = rows * D * (size + 1) + case["T"] * (case["NQ"] + case["NKV"]) * 4
        b += case["T"] * (case["rd"] * 4 + 20) + 4 * case["B"] * case["NKV"] * D
        return dict(bytes=b, flops=rows * D * 8)
    if op == "window":
        pairs, keys = _pairs(case)
        rows = sum(_requests(case)[1]) * case["NQ"]
        return dict(bytes=keys * case["NKV"] * (2 * D + 4) + rows * (3 * D + 4), flops=4 * D * pairs * case["NQ"])
    size = 2 if case["dtype"] == "bf16" else 4
    return dict(bytes=case["R"] * (case["V"] * size + 16 + 8 * case["top"]), flops=4 * case["R"] * case["V"])


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _shape(case, blocks):
    if case["layout"] == "bsnd":
        return (blocks, BS, case["NKV"], D)
    return (blocks, case["NKV"], BS, D)


def _fill_cache(case, blocks, g):
    """Codes and key scales as the per-token quantiser leaves them for N(0, 1) rows."""
    shape = _shape(case, blocks)
    k = torch.empty(shape, dtype=torch.uint8, device="cuda")
    v = torch.empty(shape, dtype=torch.uint8, device="cuda")
    ks = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    for i in range(0, blocks, 512):
        m = min(512, blocks - i)
        x = torch.randn((m,) + shape[1:], generator=g, device="cuda")
        s = x.abs().amax(-1) / 448
        k[i:i + m] = (x / s[..., None]).clamp(-448, 448).to(F8).view(torch.uint8)
        ks[i:i + m] = s
        x = torch.randn((m,) + shape[1:], generator=g, device="cuda")
        v[i:i + m] = (x * (448 / 4.5)).clamp(-448, 448).to(F8).view(torch.uint8)
    return k, v, ks


def _pair_axis(case):
    """The axis of each rotary pair: a quarter time, the rest height and width by
    halves, one section behind another or in turn."""
    half = case["rd"] // 2
    t, h = half // 4, (half - half // 4) // 2
    if case["axes"] == "sections":
        return [0] * t + [1] * h + [2] * (half - t - h)
    return [i % 3 for i in range(half)]


def _positions(case, g):
    """Time, height and width of each token: pieces of text, where the three are
    one, and of images, where the time stands and the others walk over a grid."""
    T = case["T"]
    i = torch.arange(T, device="cuda")
    piece = i // 96
    start = torch.randint(0, 30000, (T // 96 + 1,), generator=g, device="cuda")[piece]
    image = (torch.rand(T // 96 + 1, generator=g, device="cuda") < 0.6)[piece]
    at = i % 96
    pos = torch.stack([torch.where(image, start, start + at), torch.where(image, start + at // 12, start + at),
                       torch.where(image, start + at % 12, start + at)])
    return pos.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "plan":
        B, T = case["B"], case["T"]
        ctx, new = _requests(case)
        r = random.Random(seed)
        r.shuffle(ctx)
        width = (case["hi"] + T + BS - 1) // BS + 1
        held = [(c + BS - 1) // BS for c in ctx]
        fresh = sum((c + n + BS - 1) // BS for c, n in zip(ctx, new)) - sum(held)
        ids = list(range(sum(held) + fresh + 9))
        r.shuffle(ids)
        rows, at = [], 0
        for m in held:
            rows.append(ids[at:at + m] + [-1] * (width - m))
            at += m
        # a few blocks at the pool's begin are taken already; it runs out in one seed of four
        st["head"] = _i32([5])
        st["pool"] = _i32(ids[:5] + ids[at:at + fresh + (4 if seed % 4 else -(fresh // 8))])
        st["blocks"] = len(ids)
        st["act"], st["lens"], st["bt"] = _i32(ctx), _i32(new), _i32(rows)
        for name, n in (("slots", T), ("pos", T), ("tb", T), ("cu", B + 1), ("new_act", B), ("new_head", 1)):
            st[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
        if own:
            st["call"] = _pa().prepare_plan_batch(
                st["act"], st["lens"], st["pool"], st["head"], st["bt"], st["slots"], st["pos"], st["tb"], st["cu"],
                st["new_act"], st["new_head"], num_blocks=st["blocks"])
    elif op == "append":
        T, NQ, NKV, B = case["T"], case["NQ"], case["NKV"], case["B"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        qkv = torch.randn((T, (NQ + 2 * NKV) * D), generator=g, device="cuda").to(dt)
        st["q"] = qkv[:, :NQ * D].view(T, NQ, D)
        st["k"] = qkv[:, NQ * D:(NQ + NKV) * D].view(T, NKV, D)
        st["v"] = qkv[:, (NQ + NKV) * D:].view(T, NKV, D)
        st["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        st["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        ang = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * torch.exp(
            torch.arange(case["rd"] // 2, dtype=torch.float64, device="cuda") * (-math.log(1e6) * 2 / case["rd"]))
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        st["pos"] = _positions(case, g)
        st["axis"] = torch.tensor(_pair_axis(case), device="cuda")
        st["tb"] = torch.randint(0, B, (T,), generator=g, device="cuda", dtype=torch.int32)
        st["vs"] = (2.5 + 2 * torch.rand((B, NKV, D), generator=g, device="cuda")) / 448
        blocks = (T + BS - 1) // BS + 2
        slots = torch.randperm(blocks * BS, generator=g, device="cuda")[:T].to(torch.int32)
        slots[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
        st["slots"] = slots
        shape = _shape(case, blocks)
        st["kc"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        st["ksc"] = torch.zeros(shape[:3], dtype=torch.float32, device="cuda")
        st["qc"] = torch.zeros((T, NQ, D), dtype=torch.uint8, device="cuda")
        st["qs"] = torch.zeros((T, NQ), dtype=torch.float32, device="cuda")
        if own:
            pa = _pa()
            st["call"] = pa.prepare_qkv_norm_mrope_append(
                st["q"], st["k"], st["v"], st["qw"], st["kw"], st["cos_sin"], st["pos"], st["qc"], st["qs"], st["kc"],
                st["vc"], st["slots"], st["ksc"], st["vs"], st["tb"], pair_axis=_pair_axis(case), eps=1e-5,
                interleaved=case["inter"], layout=pa.LAYOUT_BSND if case["layout"] == "bsnd" else pa.LAYOUT_BNBD)
    elif op == "window":
        B, NQ, NKV = case["B"], case["NQ"], case["NKV"]
        ctx, new = _requests(case)
        r = random.Random(seed)
        act = [c + n for c, n in zip(ctx, new)]
        # the first tokens' blocks and those that a token's window reaches; the others
        # have been given back: -1
        need = [sorted(set(range(min(-(-case["sinks"] // BS), -(-a // BS)))) |
                       set(range(max(0, c - case["window"] + 1) // BS, -(-a // BS)))) for c, a in zip(ctx, act)]
        total = sum(map(len, need))
        blocks = total + total // 10 + 1
        ids = list(range(blocks))
        r.shuffle(ids)
        width = max(-(-a // BS) for a in act)
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = torch.tensor([b for b in range(B) for _ in need[b]]), torch.tensor([i for m in need for i in m])
        table[at] = torch.tensor(ids[:total], dtype=torch.int32)
        st["bt"] = table.cuda()
        st["kc"], st["vc"], st["ksc"] = _fill_cache(case, blocks, g)
        T = sum(new)
        x = torch.randn((T, NQ, D), generator=g, device="cuda")
        st["qs"] = x.abs().amax(-1) / 448
        st["qc"] = (x / st["qs"][..., None]).clamp(-448, 448).to(F8).view(torch.uint8)
        st["vs"] = (4 + torch.rand((B, NKV, D), generator=g, device="cuda")) / 448
        st["act"], st["cu"] = _i32(act), _i32([sum(new[:b]) for b in range(B + 1)])
        st["out"] = torch.empty((T, NQ, D), dtype=torch.bfloat16, device="cuda")
        if own:
            pa = _pa()
            st["ws"] = pa.WindowWorkspace(case["most"], NQ, NKV)
            st["call"] = pa.prepare_window_attention(
                st["qc"], st["qs"], st["kc"], st["ksc"], st["vc"], st["vs"], st["bt"], st["act"], st["cu"], st["out"],
                window=case["window"], sinks=case["sinks"], max_tokens=case["most"], workspace=st["ws"],
                layout=pa.LAYOUT_BSND if case["layout"] == "bsnd" else pa.LAYOUT_BNBD)
    else:
        R, V, top = case["R"], case["V"], case["top"]
        # rows of a projection whose vocabulary is padded
        x = torch.empty((R, V + case["pad"]), dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32,
                        device="cuda")
        for i in range(0, R, 256):
            m = min(256, R - i)
            x[i:i + m] = 3 * torch.randn((m, V + case["pad"]), generator=g, device="cuda")
        st["x"] = x[:, :V]
        # a drawn token mostly, one with a masked logit now and then
        st["tok"] = torch.empty(R, dtype=torch.int32, device="cuda")
        for i in range(0, R, 256):
            p = torch.softmax(st["x"][i:i + 256].float(), -1)
            st["tok"][i:i + 256] = torch.multinomial(p, 1, generator=g)[:, 0].int()
        masked = torch.randint(0, V, (R, 16), generator=g, device="cuda")
        x.scatter_(1, masked[:, :8], -math.inf)
        for name, shape, dt in (("lp", (R,), torch.float32), ("rank", (R,), torch.int32), ("ent", (R,), torch.float32),
                                ("tid", (R, top), torch.int32), ("tlp", (R, top), torch.float32)):
            st[name] = torch.zeros(shape, dtype=dt, device="cuda")
        if own:
            st["call"] = _pa().prepare_token_logprobs(
                st["x"], st["tok"], st["lp"], ranks=st["rank"], entropy=st["ent"],
                top_ids=st["tid"] if top else None, top_logprobs=st["tlp"] if top else None)
    return st


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _plan(st):
    act, new, pool, bt = st["act"].long(), st["lens"].long(), st["pool"].long(), st["bt"]
    T, width = st["slots"].shape[0], bt.shape[1]
    head = st["head"].long()
    held = (act + BS - 1) // BS
    cum = torch.cumsum(new, 0)
    fits = (act + new <= width * BS) & (cum <= T)
    need = torch.where(fits, (act + new + BS - 1) // BS - held, 0)
    end = torch.cumsum(need, 0)
    fits = fits & ((need == 0) | (head + end <= pool.shape[0]))
    new_head = head + torch.where(fits & (need > 0), end, 0).amax()
    # the new blocks' entries
    j = torch.arange(width, device="cuda")[None]
    k = j - held[:, None]
    take = fits[:, None] & (k >= 0) & (k < need[:, None])
    source = (head + end[:, None] - need[:, None] + k).clamp(0, pool.shape[0] - 1)
    bt.copy_(torch.where(take, pool[source], bt.long()))
    # the tokens
    cu = torch.cat([torch.zeros_like(cum[:1]), cum.clamp(max=T)])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = t < cu[-1]
    b = torch.where(real, b, 0)
    pos = torch.where(real, act[b] + t - cu[b], 0)
    block = bt[b, (pos // BS).clamp(max=width - 1)].long()
    ok = real & fits[b] & (block >= 0) & (block < st["blocks"])
    slots = torch.where(ok, block * BS + pos % BS, -1)
    return [bt, slots.int(), pos.int(), b.int(), cu.int(), torch.where(fits, act + new, act).int(), new_head.int()]


def _norm_rope(x, w, c, s, inter, eps):
    """RMSNorm over the last axis, weight, rotation by each pair's angle."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    half = c.shape[-1]
    c, s = c[:, None], s[:, None]
    if inter:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _quant(y):
    s = y.abs().amax(-1) / 448
    return (y / torch.where(s == 0, 1, s)[..., None]).clamp(-448, 448), s


def _place(case, cache, slots, rows):
    """rows [T, NKV, ...] to the cache's slots; the others of the cache stay."""
    ok = slots >= 0
    s = slots[ok].long()
    if case["layout"] == "bsnd":
        cache[s // BS, s % BS] = rows[ok]
    else:
        cache[s // BS, :, s % BS] = rows[ok]


def _append(st):
    case = st["case"]
    half = case["rd"] // 2
    pair = torch.arange(half, device="cuda")
    at = st["pos"].long()[st["axis"]].T                    # [T, pairs]
    c, s = st["cos_sin"][at, pair], st["cos_sin"][at, half + pair]
    qn, qs = _quant(_norm_rope(st["q"], st["qw"], c, s, case["inter"], 1e-5))
    kn, ks = _quant(_norm_rope(st["k"], st["kw"], c, s, case["inter"], 1e-5))
    vn = (st["v"].float() / st["vs"][st["tb"].long()]).clamp(-448, 448)
    _place(case, st["kc"], st["slots"], kn.to(F8).view(torch.uint8))
    _place(case, st["vc"], st["slots"], vn.to(F8).view(torch.uint8))
    _place(case, st["ksc"], st["slots"], ks)
    return [qn.to(F8), qs, st["kc"].view(F8), st["vc"].view(F8), st["ksc"]]


def _rows_at(st, name, pos):
    """[B, NKV, positions, ...] float of the cache's rows at positions [B, L]."""
    bt = st["bt"]
    block = torch.gather(bt, 1, (pos // BS).clamp(max=bt.shape[1] - 1)).clamp(min=0).long()
    c = st[name]
    x = c[block, pos % BS] if st["case"]["layout"] == "bsnd" else c[block, :, pos % BS]
    x = x.transpose(1, 2)
    return x.view(F8).float() if x.dtype == torch.uint8 else x


def _window(st):
    """All sequences at once, padded; long ones some tokens at a time."""
    case = st["case"]
    NQ, NKV, W, S = case["NQ"], case["NKV"], case["window"], case["sinks"]
    G, act, cu = NQ // NKV, st["act"].long(), st["cu"].long()
    n = cu[1:] - cu[:-1]
    ctx, B = act - n, case["B"]
    out = torch.zeros((st["qc"].shape[0], NQ, D), device="cuda")
    # scores of 2^30 (row, key) pairs at most
    step = case["most"]
    while step > 1 and B * NQ * step * (S + W + step) > 1 << 30:
        step = (step + 1) // 2
    for i0 in range(0, case["most"], step):
        i = i0 + torch.arange(step, device="cuda")[None]
        real = i < n[:, None]                              # [B, tokens]
        row = (cu[:-1, None] + i).clamp(max=out.shape[0] - 1)
        p = ctx[:, None] + i
        lo = (ctx + i0 - W + 1).clamp(min=0)
        near = lo[:, None] + torch.arange(W - 1 + step, device="cuda")[None]
        first = torch.arange(S, device="cuda")[None].expand(B, S)
        pos = torch.cat([first, near], 1)                  # [B, keys]
        seen = (pos[:, None] <= p[:, :, None]) & torch.cat(
            [torch.ones_like(first, dtype=torch.bool)[:, None].expand(B, step, S),
             (near >= S)[:, None] & (near[:, None] > p[:, :, None] - W)], 2)
        at = pos.clamp(max=st["bt"].shape[1] * BS - 1)
        k = _rows_at(st, "kc", at) * _rows_at(st, "ksc", at)[..., None]
        q = st["qc"][row].view(F8).float() * st["qs"][row][..., None]
        q = q.view(B, step, NKV, G, D).permute(0, 2, 1, 3, 4).reshape(B, NKV, step * G, D)
        s = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D)
        s = s.view(B, NKV, step, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf).flatten(2, 3)
        s = torch.exp_(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)))
        total = s.sum(-1, keepdim=True)
        o = torch.matmul(s, _rows_at(st, "vc", at)) * st["vs"][:, :, None]
        o = torch.where(total > 0, o / total, 0)
        o = o.view(B, NKV, step, G, D).permute(0, 2, 1, 3, 4).reshape(B, step, NQ, D)
        out[row[real]] = o[real]
    return out.to(torch.bfloat16)


def _logp(st):
    x, top = st["x"].float(), st["case"]["top"]
    tok = st["tok"].long()[:, None]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    logz = m + torch.log(total)
    own_x = torch.gather(x, 1, tok)
    rank = (x > own_x).sum(-1).int()
    ent = (torch.log(total) - (e * torch.where(e > 0, x - m, 0)).sum(-1, keepdim=True) / total)[:, 0]
    lp = (own_x - logz)[:, 0]
    if top == 0:
        return [lp, rank, ent]
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    return [lp, rank, ent, i[:, :top].int(), v[:, :top] - logz]


def run(st):
    op = st["case"]["op"]
    if own:
        st["call"]()
        if op == "plan":
            return [st["bt"], st["slots"], st["pos"], st["tb"], st["cu"], st["new_act"], st["new_head"]]
        if op == "append":
            return [st["qc"].view(F8), st["qs"], st["kc"].view(F8), st["vc"].view(F8), st["ksc"]]
        if op == "window":
            return st["out"]
        return [st["lp"], st["rank"], st["ent"]] + ([st["tid"], st["tlp"]] if st["case"]["top"] else [])
    return {"plan": _plan, "append": _append, "window": _window, "logp": _logp}[op](st)


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------

def _exact_plan(st):
    """Request by request and token by token."""
    act, new, pool, bt = (st[k].tolist() for k in ("act", "lens", "pool", "bt"))
    T, width, taken = st["slots"].shape[0], st["bt"].shape[1], 0
    head = last = int(st["head"][0])
    cu, new_act, slots, pos, batch = [0], [], [-1] * T, [0] * T, [0] * T
    rows = 0
    for b, (a, n) in enumerate(zip(act, new)):
        rows += n
        ok = a + n <= width * BS and rows <= T
        have, need = -(-a // BS), -(-(a + n) // BS) - -(-a // BS) if ok else 0
        if need:
            taken += need
            ok = head + taken <= len(pool)
            if ok:
                bt[b][have:have + need] = pool[head + taken - need:head + taken]
                last = head + taken
        for t in range(cu[-1], min(rows, T)):
            p = a + t - cu[-1]
            batch[t], pos[t] = b, p
            block = bt[b][p // BS] if ok else -1
            slots[t] = block * BS + p % BS if 0 <= block < st["blocks"] else -1
        cu.append(min(rows, T))
        new_act.append(a + n if ok else a)
    return [_i32(v) for v in (bt, slots, pos, batch, cu, new_act, [last])]


def _exact_append(st):
    case = st["case"]
    T, rd = case["T"], case["rd"]
    half = rd // 2
    table = st["cos_sin"].double()
    cos = torch.stack([table[st["pos"][a].long(), i] for i, a in enumerate(_pair_axis(case))], -1)[:, None]
    sin = torch.stack([table[st["pos"][a].long(), half + i] for i, a in enumerate(_pair_axis(case))], -1)[:, None]
    idx = torch.arange(half, device="cuda")
    ia, ib = (2 * idx, 2 * idx + 1) if case["inter"] else (idx, idx + half)
    res = []
    for name, w in (("q", "qw"), ("k", "kw")):
        x = st[name].double()
        y = x / ((x ** 2).sum(-1, keepdim=True) / D + 1e-5).sqrt() * st[w].double()
        z = y.clone()
        z[..., ia] = y[..., ia] * cos - y[..., ib] * sin
        z[..., ib] = y[..., ia] * sin + y[..., ib] * cos
        scale = z.abs().max(-1).values / 448
        # the codes' own precision is eight bits: the values before they are rounded
        res.append((z / scale[..., None], scale))
    qn, qs = res[0]
    kn, ks = res[1]
    vn = (st["v"].double() / st["vs"].double()[st["tb"].long()]).clamp(-448, 448)
    shape = st["kc"].shape
    flat = torch.arange(T, device="cuda")[st["slots"] >= 0]
    s = st["slots"].long()[flat]
    outs = []
    for rows, tail in ((kn, (D,)), (vn, (D,)), (ks, ())):
        c = torch.zeros(tuple(shape[:3]) + tail, dtype=torch.float64, device="cuda")
        if case["layout"] == "bnbd":
            c = c.transpose(1, 2)
        c[s // BS, s % BS] = rows[flat]
        outs.append(c.transpose(1, 2).contiguous() if case["layout"] == "bnbd" else c)
    return [qn, qs, outs[0], outs[1], outs[2]]


def _exact_window(st):
    """One sequence and kv head at a time, over the positions any of its tokens sees."""
    case = st["case"]
    NQ, NKV = case["NQ"], case["NKV"]
    G = NQ // NKV
    out = torch.zeros((st["qc"].shape[0], NQ, D), dtype=torch.float64, device="cuda")
    ctx, new = _requests(case)
    row = 0
    for b in range(case["B"]):
        for i0 in range(0, new[b], 1024):
            m = min(1024, new[b] - i0)
            p = torch.arange(ctx[b] + i0, ctx[b] + i0 + m, device="cuda")
            at = torch.arange(0, ctx[b] + i0 + m, device="cuda")
            at = at[(at < case["sinks"]) | (at > ctx[b] + i0 - case["window"])]
            far = p[:, None] - at[None]
            see = (far >= 0) & ((far < case["window"]) | (at[None] < case["sinks"]))
            blk, off = st["bt"][b].long()[at // BS], at % BS
            for h in range(NKV):
                ix = (blk, off, h) if case["layout"] == "bsnd" else (blk, h, off)
                k = st["kc"][ix].view(F8).double() * st["ksc"][ix].double()[:, None]
                v = st["vc"][ix].view(F8).double() * st["vs"][b, h].double()
                hs, rs = slice(h * G, (h + 1) * G), slice(row + i0, row + i0 + m)
                q = st["qc"][rs, hs].view(F8).double() * st["qs"][rs, hs, None].double()
                a = (q.reshape(m * G, D) @ k.T * D ** -0.5).view(m, G, -1)
                a = torch.where(see[:, None], a, -math.inf)
                a = torch.exp(a - a.max(-1, keepdim=True).values)
                a = a / a.sum(-1, keepdim=True)
                out[rs, hs] = (a.view(m * G, -1) @ v).view(m, G, D)
        row += new[b]
    return out


def _exact_logp(st):
    R, V = st["x"].shape
    top = st["case"]["top"]
    outs = [[], [], [], [], []]
    for i in range(0, R, 128):
        x = st["x"][i:i + 128].double()
        t = st["tok"][i:i + 128].long()
        logp = x - torch.logsumexp(x, -1, keepdim=True)
        at = torch.arange(x.shape[0], device="cuda")
        outs[0].append(logp[at, t])
        outs[1].append(torch.sum(x > x[at, t][:, None], -1).int())
        outs[2].append(-torch.nansum(torch.exp(logp) * logp, -1))
        order = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :top]
        outs[3].append(order.int())
        outs[4].append(torch.gather(logp, 1, order))
    outs = [torch.cat(o) for o in outs]
    return outs if top else outs[:3]


def exact(case, seed):
    if case["op"] == "window" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "window": _exact_window, "logp": _exact_logp}[case["op"]](st)
