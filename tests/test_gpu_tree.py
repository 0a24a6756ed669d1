"""The speculative decode step's operators on the GPU against plain 64-bit
forms: attention of a drafted tree, norm + rotation + quantising append,
verification, the accepted branch in the cache, and a run of them together."""
import numpy as np
import pytest

from tests import _draft_helpers as H

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_paged_kv_block_gb300 as pa
    return pa


def _cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def run_tree(c, ws=None, mask=None, use_len=True, out=None, scale=None, stream=None):
    pa = _pa()
    g = _cuda(c)
    if out is None:
        out = torch.full((c["B"] * c["S1"], c["NQ"], H.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = ws or pa.TreeWorkspace(c["B"], c["S1"], c["NQ"], c["NKV"])
    pa.tree_decode(g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"],
                   g["mask"] if mask is None else mask, out, S1=c["S1"],
                   tree_len=g["n"] if use_len else None, layout=c["layout"], workspace=ws,
                   softmax_scale=scale, stream=stream)
    torch.cuda.synchronize()
    assert ws.error_flags() == 0
    return out


def check_tree(c, out, scale=None):
    ref, tol = H.tree_reference(c, scale)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() - tol).max()),
                           [tuple(int(i) for i in x) for x in bad.nonzero()[:4]])


TREES = [
    # ctx, S1, NQ, NKV, layout, n
    ([5], 1, 1, 1, 0, None),                       # one row of one head
    ([0], 1, 12, 1, 1, None),                      # nothing but itself
    ([0, 1, 127, 128, 129], 4, 8, 2, 0, None),     # around a block's end
    ([300, 37, 511], 8, 4, 1, 1, [8, 3, 0]),       # ragged trees, one of them empty
    ([250, 1000], 5, 96, 8, 0, None),              # group of 12
    ([700, 90], 16, 12, 1, 1, [16, 11]),           # 192 rows a kv head
    ([1300], 64, 48, 8, 0, None),                  # 384 rows
    ([257, 120], 128, 2, 1, 1, [128, 77]),         # the most drafted tokens, two tiles of them
    ([60], 3, 128, 1, 0, None),                    # the largest group
    ([130, 1, 640, 383, 4, 2000, 77], 7, 15, 3, 1, [7, 1, 6, 0, 4, 7, 5]),
]


@pytest.mark.parametrize("i", range(len(TREES)))
def test_tree_decode_matches_64_bit(i):
    ctx, S1, NQ, NKV, layout, n = TREES[i]
    c = H.tree_case(100 + i, ctx, S1, NQ, NKV, layout, n=n, room=i % 3)
    check_tree(c, run_tree(c))


@pytest.mark.parametrize("layout", [0, 1])
def test_tree_decode_long_context_is_split_and_joined(layout):
    c = H.tree_case(7, [20000, 3], 4, 12, 1, layout)
    check_tree(c, run_tree(c))


def test_tree_decode_many_sequences():
    rng = np.random.default_rng(3)
    ctx = [int(x) for x in rng.integers(0, 400, 200)]
    n = [int(x) for x in rng.integers(0, 6, 200)]
    c = H.tree_case(8, ctx, 5, 8, 2, 0, n=n)
    check_tree(c, run_tree(c))


def test_tree_decode_rows_without_keys_and_foreign_masks():
    """A mask that leaves rows empty (no context, no node), one that sees later
    nodes, and one for all sequences: any mask is taken as it is."""
    c = H.tree_case(11, [0, 140, 0], 6, 12, 2, 0)
    c["mask"][0, 2] = False
    c["mask"][1, 3] = False
    c["mask"][1, 0, 5] = True
    c["mask"][2] = False
    out = run_tree(c)
    check_tree(c, out)
    assert (out[2] == 0).all() and (out[12:] == 0).all()
    shared = H.ancestor_mask([-1, 0, 0, 1, 1, 2])
    c["mask"] = torch.from_numpy(shared)[None].expand(3, 6, 6)
    out = run_tree(c, mask=torch.from_numpy(shared).cuda())
    check_tree(c, out)


def test_tree_decode_ignores_what_lies_behind_the_sequence():
    """NaN codes and NaN or infinite key scales past the length, in the same
    page, and in blocks that no sequence holds."""
    c = H.tree_case(12, [200, 77], 5, 16, 4, 0, room=2)
    clean = run_tree(c).clone()
    kc, vc, ks = (H.by_position(c[k], 0) for k in ("kc", "vc", "ks"))
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b in range(2):
        pos = torch.arange(int(c["act"][b]))
        used[c["bt"][b].long()[pos // 128], pos % 128] = True
    kc[~used] = 0x7F
    vc[~used] = 0xFF
    ks[~used] = float("nan")
    ks[:, 127][~used[:, 127]] = float("inf")
    assert torch.equal(run_tree(c), clean)


def test_tree_decode_extreme_scores_and_outliers():
    """Scores of hundreds (one key takes all), a key that outweighs the rest by
    2^20, and equal keys."""
    c = H.tree_case(13, [1500, 260, 129], 3, 8, 2, 1)
    ks = H.by_position(c["ks"], 1)
    ks[:, ::64] *= 40.0
    check_tree(c, run_tree(c))
    kc = H.by_position(c["kc"], 1)
    kc[:] = kc[0, 0, 0]
    c["ks"][:] = 0.01
    check_tree(c, run_tree(c))


def test_tree_decode_bad_block_ids_read_block_zero_and_lengths_are_clamped():
    c = H.tree_case(14, [300, 40], 4, 4, 1, 0)
    c["bt"][0, 1] = -1
    c["bt"][1, 0] = 10 ** 6
    c["act"][0] = 10 ** 6                 # past the table: clamped to its capacity
    check_tree(c, run_tree(c))
    c["act"][0] = -5
    c["act"][1] = 2                       # fewer than the drafted tokens
    check_tree(c, run_tree(c))


def test_tree_decode_scale_and_all_drafted_tokens_by_default():
    c = H.tree_case(15, [333, 18], 6, 8, 1, 0)
    check_tree(c, run_tree(c, use_len=False, scale=0.02), 0.02)
    check_tree(c, run_tree(c, scale=-0.05), -0.05)


def test_tree_decode_is_repeatable_bit_for_bit():
    c = H.tree_case(16, [9000, 1], 8, 24, 2, 0)
    pa = _pa()
    ws = pa.TreeWorkspace(c["B"], 8, 24, 2)
    first = run_tree(c, ws=ws).clone()
    for _ in range(3):
        assert torch.equal(run_tree(c, ws=ws), first)


def test_tree_decode_on_another_stream_and_replayed_from_a_graph():
    pa = _pa()
    c = H.tree_case(17, [500, 900], 8, 12, 1, 0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = run_tree(c)
    check_tree(c, out)
    check_tree(c, run_tree(c, stream=side))
    g = _cuda(c)
    out = torch.empty((16, 12, H.D), dtype=torch.bfloat16, device="cuda")
    ws = pa.TreeWorkspace(2, 8, 12, 1)
    with torch.cuda.stream(side):
        call = pa.prepare_tree_decode(g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"],
                                      g["mask"], out, S1=8, tree_len=g["n"], layout=0, workspace=ws)
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for act in ([508, 908], [20, 130], [0, 0]):
        c["act"] = torch.tensor(act, dtype=torch.int32)
        g["act"].copy_(c["act"])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_tree(c, out)
    assert ws.error_flags() == 0


def test_tree_decode_of_one_token_agrees_with_decode():
    """S1 = 1 over the same cache: the two decodes differ by decode()'s FP8 P."""
    pa = _pa()
    c = H.tree_case(18, [99, 700, 1], 1, 96, 8, 0)
    g = _cuda(c)
    a = run_tree(c)
    b = torch.empty_like(a)
    pa.decode(g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"], b, layout=0)
    torch.cuda.synchronize()
    ref, tol = H.tree_reference(c)
    # decode(): P rounded to E4M3, half a step 2^-4, so 2^-4 of the mass (tol >= 2^-11 of it)
    assert ((a.double() - b.double()).cpu().abs() <= tol * (1 + 2 ** 7)).all()


# ---- norm, rotation, append -----------------------------------------------------

def append_case(seed, T, NQ, NKV, D, rd, dtype, layout, B=3, strided=True, wdt=None, idt=torch.int32):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
    H3 = NQ + 2 * NKV
    qkv = t(rng.standard_normal((T, H3 * D), dtype=np.float32) * 2).to(dtype)
    q, k, v = (qkv[:, :NQ * D].view(T, NQ, D), qkv[:, NQ * D:(NQ + NKV) * D].view(T, NKV, D),
               qkv[:, (NQ + NKV) * D:].view(T, NKV, D))
    ang = rng.uniform(0, 6.28, (50, max(rd // 2, 1)))
    cs = t(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)) if rd else None
    NB, BS = T // 16 + 3, 16
    slots = rng.permutation(NB * BS)[:T].astype(np.int32)
    slots[::7] = -1
    slots[1::11] = NB * BS
    c = dict(q=q, k=k, v=v, qkv=qkv, cs=cs, pos=t(rng.integers(-3, 60, T)).to(idt), slots=t(slots).to(idt),
             qw=t(1 + 0.3 * rng.standard_normal(D, dtype=np.float32)).to(wdt or dtype),
             kw=t(1 + 0.3 * rng.standard_normal(D, dtype=np.float32)).to(wdt or dtype),
             vs=t(rng.uniform(0.01, 0.03, (B, NKV, D)).astype(np.float32)),
             tb=t(rng.integers(0, B, T).astype(np.int32)), NB=NB, BS=BS, layout=layout, D=D)
    return c


def run_append(c, eps=1e-5, inter=False, norm=True, strided=True):
    pa = _pa()
    T, NQ, D = c["q"].shape
    NKV = c["k"].shape[1]
    sh = (c["NB"], c["BS"], NKV) if c["layout"] == 0 else (c["NB"], NKV, c["BS"])
    kc = torch.full(sh + (D,), 0xA5, dtype=torch.uint8, device="cuda")
    vc = torch.full(sh + (D,), 0x5A, dtype=torch.uint8, device="cuda")
    ks = torch.full(sh, -7.0, device="cuda")
    qc = torch.zeros((T, NQ, D), dtype=torch.uint8, device="cuda")
    qs = torch.zeros((T, NQ), device="cuda")
    qkv = c["qkv"].cuda()
    q, k, v = (qkv[:, :NQ * D].view(T, NQ, D), qkv[:, NQ * D:(NQ + NKV) * D].view(T, NKV, D),
               qkv[:, (NQ + NKV) * D:].view(T, NKV, D))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pa.qkv_norm_rope_append(q, k, v, c["qw"].cuda() if norm else None, c["kw"].cuda() if norm else None,
                            c["cs"].cuda() if c["cs"] is not None else None, c["pos"].cuda(), qc, qs, kc, vc,
                            c["slots"].cuda(), ks, c["vs"].cuda(), c["tb"].cuda(), eps=eps, interleaved=inter,
                            layout=c["layout"])
    torch.cuda.synchronize()
    return tuple(x.cpu() for x in (qc, qs, kc, vc, ks))


def check_codes(y, code, scale, check_scale=True):
    """E4M3 codes against y: half a step (2^-4 of the value, 2^-10 where the
    code is subnormal) plus the FP32 arithmetic before them, 64 roundings of
    2^-24 of the row's maximum (448 codes). The scale is a float: below 2^-126
    its step is 2^-149 whatever its value, so half of that is added. The same
    holds of y, which is FP32 by definition: where it lies below 2^-126 each of
    the 64 roundings is half of 2^-149, or 2^-150 / scale in codes, and not 2^-24
    of it."""
    amax = y.abs().amax(-1)
    s = amax / 448
    if check_scale:
        assert ((scale.double() - s).abs() <= s * 2.0 ** -18 + 2.0 ** -150).all()
    want = y / torch.where(s == 0, 1.0, s)[..., None]
    got = H.value(code)
    tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 + 448 * 2.0 ** -18
    tol = tol + torch.where((amax > 0) & (amax < 2.0 ** -126), 64 * 2.0 ** -150 / torch.where(s == 0, 1.0, s), 0.0)[..., None]
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())


def check_append(c, got, eps=1e-5, inter=False, norm=True):
    qc, qs, kc, vc, ks = got
    y = H.norm_rope_reference(c["q"], c["qw"] if norm else None, c["cs"], c["pos"], inter, eps)
    check_codes(y, qc, qs)
    y = H.norm_rope_reference(c["k"], c["kw"] if norm else None, c["cs"], c["pos"], inter, eps)
    kc, vc, ks = (H.by_position(x, c["layout"]) for x in (kc, vc, ks))
    s = c["slots"].long()
    ok = (s >= 0) & (s < c["NB"] * c["BS"])
    blk, off = s[ok] // c["BS"], s[ok] % c["BS"]
    check_codes(y[ok], kc[blk, off], ks[blk, off])
    vsc = c["vs"][c["tb"].long()]
    # v is encoded as cache_quant_scatter encodes it: bit for bit
    v = (c["v"].float() / vsc).clamp(-448, 448).to(H.F8).view(torch.uint8)
    assert torch.equal(vc[blk, off], v[ok])
    rest = torch.ones(kc.shape[:2], dtype=torch.bool)
    rest[blk, off] = False
    assert (kc[rest] == 0xA5).all() and (vc[rest] == 0x5A).all() and (ks[rest] == -7.0).all()


APPENDS = [
    # T, NQ, NKV, D, rd, dtype, layout, inter
    (1, 1, 1, 128, 64, torch.bfloat16, 0, False),
    (16, 96, 8, 128, 64, torch.bfloat16, 1, False),
    (37, 12, 2, 128, 128, torch.float32, 0, True),
    (29, 5, 3, 64, 32, torch.bfloat16, 1, False),
    (13, 3, 1, 64, 64, torch.float32, 1, True),
    (11, 4, 2, 256, 256, torch.bfloat16, 0, False),
    (9, 7, 1, 256, 16, torch.float32, 0, False),
    (21, 2, 2, 128, 8, torch.bfloat16, 0, True),
    (50, 6, 2, 128, 0, torch.float32, 0, False),
]


@pytest.mark.parametrize("i", range(len(APPENDS)))
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_64_bit(i, norm):
    T, NQ, NKV, D, rd, dtype, layout, inter = APPENDS[i]
    c = append_case(i, T, NQ, NKV, D, rd, dtype, layout, idt=torch.int64 if i % 2 else torch.int32,
                    wdt=torch.float32 if i % 3 == 0 else torch.bfloat16)
    check_append(c, run_append(c, inter=inter, norm=norm, strided=i != 4), inter=inter, norm=norm)


def test_append_zero_tiny_and_huge_rows():
    c = append_case(40, 8, 4, 2, 128, 64, torch.float32, 0)
    c["qkv"][0] = 0
    c["qkv"][1] *= 1e-38
    c["qkv"][2] *= 1e-41
    c["qkv"][3] *= 1e18
    got = run_append(c, norm=False)
    assert (got[0][0] == 0).all() and (got[1][0] == 0).all()
    y = H.norm_rope_reference(c["q"], None, c["cs"], c["pos"], False, 0)
    check_codes(y[3:], got[0][3:], got[1][3:])
    # the subnormal rows: the scale itself has few bits, the codes stay within the largest
    assert (H.value(got[0][1:3]).abs() <= 448).all() and torch.isfinite(H.value(got[0][1:3])).all()
    check_append(c, run_append(c, eps=1e-5, norm=True), eps=1e-5, norm=True)


def test_append_without_norm_and_rotation_writes_cache_quant_scatters_values():
    pa = _pa()
    c = append_case(41, 33, 8, 4, 128, 0, torch.bfloat16, 1)
    _, _, kc, vc, ks = run_append(c, norm=False)
    k2, v2, s2 = torch.full_like(kc, 0xA5).cuda(), torch.full_like(vc, 0x5A).cuda(), torch.full_like(ks, -7.0).cuda()
    pa.cache_quant_scatter(c["k"].contiguous().cuda(), c["v"].contiguous().cuda(), k2, v2, c["slots"].cuda(), s2,
                           c["vs"].cuda(), c["tb"].cuda(), layout=1)
    assert torch.equal(vc, v2.cpu()) and torch.equal(ks, s2.cpu())
    # the keys' codes may differ by the reciprocal's rounding: one step at a border
    a, b = H.value(kc), H.value(k2)
    assert ((a - b).abs() <= 2.0 ** -3 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -9).all()
    assert (a != b).double().mean() < 1e-3


# ---- verification ---------------------------------------------------------------

def verify_case(seed, B, S1, V, draft, peaked=2.0, width=3):
    rng = np.random.default_rng(seed)

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)
    x = rng.standard_normal((B, S1, V)) * peaked
    q = soft(x)
    p = soft(x + 0.5 * rng.standard_normal((B, S1, V)))
    par = np.array([H.random_tree(rng, S1, width) for _ in range(B)], np.int32)
    tok = np.zeros((B, S1), np.int32)
    for b in range(B):
        for s in range(1, S1):
            tok[b, s] = rng.choice(V, p=q[b, par[b, s]].astype(np.float64) / q[b, par[b, s]].astype(np.float64).sum())
    u = rng.random((B, S1), dtype=np.float32)
    n = rng.integers(0, S1 + 1, B).astype(np.int32)
    return dict(p=p, q=q if draft else None, tok=tok, par=par, u=u, n=n)


def run_verify(c):
    pa = _pa()
    B, S1, V = c["p"].shape
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    path = torch.full((B, S1), -9, dtype=torch.int32, device="cuda")
    tokens = torch.full((B, S1), -9, dtype=torch.int32, device="cuda")
    pa.tree_verify(t(c["p"]), t(c["q"]), t(c["tok"]), t(c["par"]), t(c["u"]), acc, path, tokens, tree_len=t(c["n"]))
    torch.cuda.synchronize()
    return acc.cpu().numpy(), path.cpu().numpy(), tokens.cpu().numpy()


def check_verify(c):
    got = run_verify(c)
    want = H.verify_reference(c["p"], c["q"], c["tok"], c["par"], c["u"], c["n"])
    for g, w, name in zip(got, want, ("accepted", "path", "tokens")):
        assert np.array_equal(g, w), (name, g, w)
    return got


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,S1,V", [(1, 1, 1), (3, 1, 33), (5, 6, 7), (9, 8, 1000), (4, 16, 4097), (2, 5, 70001),
                                    (40, 12, 129), (2, 64, 512)])
def test_verify_matches_the_definition(B, S1, V, draft):
    check_verify(verify_case(B * 1000 + V, B, S1, V, draft, peaked=4.0 if V < 100 else 2.0))


def test_verify_largest_vocabulary():
    check_verify(verify_case(1, 1, 3, 262144, True))


@pytest.mark.parametrize("draft", [True, False])
def test_verify_edges(draft):
    """One-hot targets, drafts that cannot be accepted, repeated siblings, tokens
    outside the vocabulary, parents that are no lower index, empty rows, and
    random numbers at both ends."""
    c = verify_case(5, 12, 7, 300, draft)
    c["n"][:] = 7
    c["p"][0] = 0
    c["p"][0, :, 17] = 1
    c["tok"][0, 1:] = 17                      # every draft is the target's token
    c["p"][1] = 0
    c["p"][1, :, 5] = 1
    c["tok"][1, 1:] = 6                       # none is
    c["tok"][2, 1:] = c["tok"][2, 1]          # the same token again and again
    c["par"][2, 1:] = 0
    c["tok"][3, 2], c["tok"][3, 3] = -1, 300
    c["par"][4, 2], c["par"][4, 3], c["par"][4, 4] = 2, 6, -4
    c["p"][5] = 0                             # no mass at all: token -1
    c["u"][6] = 0
    c["u"][7] = np.float32(1) - np.float32(2.0 ** -24)
    if draft:
        c["q"][8] = c["p"][8]                 # equal distributions: always accepted
        c["q"][9] = 2.0                       # the rest is empty at once
        c["par"][9, 1:] = 0
        c["u"][9, 1:] = 0.9999
        c["q"][10, :, ::3] = 0
    c["p"][11, :, ::2] = np.float32("nan")
    c["tok"][11, 1:] |= 1                     # (no test at a NaN)
    check_verify(c)


def test_verify_follows_the_target_distribution():
    """Over many independent sequences of one tree the first new token is
    distributed as the target's row 0, whatever was drafted. 20000 draws of 8
    tokens: chi-squared with 7 degrees of freedom, its 1 - 1e-6 quantile 40.5."""
    rng = np.random.default_rng(9)
    B, S1, V = 20000, 4, 8
    p0 = rng.dirichlet(np.ones(V)).astype(np.float32)
    q0 = rng.dirichlet(np.ones(V)).astype(np.float32)
    p = np.broadcast_to(p0, (B, S1, V)).copy()
    for draft in (True, False):
        tok = rng.choice(V, size=(B, S1), p=q0.astype(np.float64) / q0.astype(np.float64).sum()).astype(np.int32)
        if not draft:
            tok[:] = np.array([0, 3, 1, 6], np.int32)
        c = dict(p=p, q=np.broadcast_to(q0, (B, S1, V)).copy() if draft else None, tok=tok,
                 par=np.broadcast_to(np.array([-1, 0, 0, 0], np.int32), (B, S1)).copy(),
                 u=rng.random((B, S1), dtype=np.float32), n=np.full(B, S1, np.int32))
        first = run_verify(c)[2][:, 0]
        count = np.bincount(first, minlength=V)
        want = p0.astype(np.float64) / p0.astype(np.float64).sum() * B
        assert ((count - want) ** 2 / want).sum() < 40.5


# ---- the accepted branch ----------------------------------------------------------

def keep_case(seed, ctx, S1, NKV, layout, D=128, BS=128):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    n = rng.integers(1, S1 + 1, B).astype(np.int32)
    acc = np.array([rng.integers(0, m + 1) for m in n], np.int32)
    path = np.full((B, S1), -1, np.int32)
    for b in range(B):
        if acc[b]:
            path[b, :acc[b]] = [0] + sorted(rng.choice(np.arange(1, n[b]), acc[b] - 1, replace=False))
    act = (np.asarray(ctx) + n).astype(np.int32)
    need = [max(1, -(-int(a) // BS)) for a in act]
    bt, NB = H.tables(rng, need, max(need) + 1)
    sh = (NB, BS, NKV) if layout == 0 else (NB, NKV, BS)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
    return dict(kc=t(rng.integers(0, 256, sh + (D,), dtype=np.uint8)), vc=t(rng.integers(0, 256, sh + (D,), dtype=np.uint8)),
                ks=t(rng.random(sh, dtype=np.float32)), bt=t(bt), act=t(act), n=t(n), path=t(path), acc=t(acc),
                layout=layout, BS=BS)


def keep_reference(c):
    kc, vc, ks = (H.by_position(c[k].clone(), c["layout"]) for k in ("kc", "vc", "ks"))
    new = []
    for b in range(len(c["act"])):
        act, n, m = (int(c[k][b]) for k in ("act", "n", "acc"))
        act = max(act, 0)
        n = min(max(n, 0), c["path"].shape[1], act)
        m = min(max(m, 0), n)
        for i in range(m):
            s = int(c["path"][b, i])
            if not 0 <= s < n:
                continue
            at = []
            for x in (act - n + s, act - n + i):
                bi = x // c["BS"]
                at.append((int(c["bt"][b, bi]) if bi < c["bt"].shape[1] else -1, x % c["BS"]))
            if any(not 0 <= a[0] < kc.shape[0] for a in at):
                continue
            for x in (kc, vc, ks):
                x[at[1][0], at[1][1]] = x[at[0][0], at[0][1]]
        new.append(act - n + m)
    return kc, vc, ks, torch.tensor(new, dtype=torch.int32)


def run_keep(c):
    pa = _pa()
    g = _cuda(c)
    new = torch.full((len(c["act"]),), -9, dtype=torch.int32, device="cuda")
    pa.cache_keep_path(g["kc"], g["vc"], g["ks"], g["bt"], g["act"], g["path"], g["acc"], new, tree_len=g["n"],
                       layout=c["layout"])
    torch.cuda.synchronize()
    return tuple(H.by_position(g[k].cpu(), c["layout"]) for k in ("kc", "vc", "ks")) + (new.cpu(),)


def check_keep(c):
    for g, w in zip(run_keep(c), keep_reference(c)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("ctx,S1,NKV,D,BS", [([0], 1, 1, 128, 128), ([0, 5, 120, 127, 128], 12, 8, 128, 128),
                                             ([1000, 3], 64, 3, 64, 16), ([40] * 30, 30, 17, 128, 128),
                                             ([100, 7], 300, 2, 256, 32), ([9], 1024, 1, 16, 16)])
def test_keep_path(ctx, S1, NKV, D, BS, layout):
    check_keep(keep_case(S1 + NKV, ctx, S1, NKV, layout, D, BS))


def test_keep_path_bad_ids_lengths_and_nodes():
    c = keep_case(3, [100, 250, 0, 30], 20, 2, 0)
    c["bt"][0, 0] = -1
    c["bt"][1, 1] = 10 ** 6
    c["acc"][2] = 50
    c["path"][3, 1] = 19
    c["n"][3] = 15
    c["act"][2] = -3
    check_keep(c)


# ---- a run of them together -------------------------------------------------------

@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_step(layout, graph):
    """append -> tree attention -> verification -> accepted branch, twice: the
    cache then holds what an append of the accepted tokens alone leaves."""
    pa = _pa()
    rng = np.random.default_rng(77 + layout)
    B, S1, NQ, NKV, V = 4, 6, 16, 2, 500
    T = B * S1
    ctx = [0, 126, 250, 40]
    width = 4
    bt_np, NB = H.tables(rng, [width] * B, width)
    sh = H.cache_shape(layout, NB, NKV)
    dev = dict(device="cuda")
    kc, vc, ks = H.codes(rng, sh + (128,)).cuda(), H.codes(rng, sh + (128,)).cuda(), torch.full(sh, 0.01, **dev)
    bt = torch.from_numpy(bt_np).cuda()
    act = torch.zeros(B, dtype=torch.int32, **dev)
    new_act = torch.tensor(ctx, dtype=torch.int32, **dev)
    n = torch.tensor([6, 4, 6, 1], dtype=torch.int32, **dev)
    qkv = torch.zeros((T, (NQ + 2 * NKV) * 128), dtype=torch.bfloat16, **dev)
    q, k, v = (qkv[:, :NQ * 128].view(T, NQ, 128), qkv[:, NQ * 128:(NQ + NKV) * 128].view(T, NKV, 128),
               qkv[:, (NQ + NKV) * 128:].view(T, NKV, 128))
    w = torch.ones(128, dtype=torch.bfloat16, **dev)
    ang = torch.rand((600, 32), **dev) * 6
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    vs = torch.full((B, NKV, 128), 0.02, **dev)
    tb = torch.arange(B, dtype=torch.int32, **dev).repeat_interleave(S1)
    node = torch.arange(S1, dtype=torch.int32, **dev).repeat(B)
    pos = torch.zeros(T, dtype=torch.int32, **dev)
    slots = torch.zeros(T, dtype=torch.int32, **dev)
    qc, qs = torch.zeros((T, NQ, 128), dtype=torch.uint8, **dev), torch.zeros((T, NQ), **dev)
    out = torch.zeros((T, NQ, 128), dtype=torch.bfloat16, **dev)
    par_np = np.array([H.random_tree(rng, S1, 3) for _ in range(B)], np.int32)
    depth = np.zeros((B, S1), np.int32)
    for b in range(B):
        for s in range(1, S1):
            depth[b, s] = depth[b, par_np[b, s]] + 1
    par = torch.from_numpy(par_np).cuda()
    depth = torch.from_numpy(depth).cuda().view(-1)
    mask = torch.from_numpy(np.stack([H.ancestor_mask(list(p)) for p in par_np])).cuda()
    p, qd = torch.zeros((B, S1, V), **dev), torch.zeros((B, S1, V), **dev)
    tok, u = torch.zeros((B, S1), dtype=torch.int32, **dev), torch.zeros((B, S1), **dev)
    acc = torch.zeros(B, dtype=torch.int32, **dev)
    path, toks = torch.zeros((B, S1), dtype=torch.int32, **dev), torch.zeros((B, S1), dtype=torch.int32, **dev)
    ws = pa.TreeWorkspace(B, S1, NQ, NKV)

    def step(stream=None):
        # the caller's bookkeeping, on the device: positions and slots of the nodes
        base = new_act[tb.long()]
        at = base + node
        pos.copy_(base + depth)
        slots.copy_(torch.where(node < n[tb.long()], bt[tb.long(), (at // 128).long()] * 128 + at % 128, -1))
        act.copy_(new_act + n)
        pa.qkv_norm_rope_append(q, k, v, w, w, cs, pos, qc, qs, kc, vc, slots, ks, vs, tb, layout=layout)
        pa.tree_decode(qc, qs, kc, ks, vc, vs, bt, act, mask, out, S1=S1, tree_len=n, layout=layout, workspace=ws)
        pa.tree_verify(p, qd, tok, par, u, acc, path, toks, tree_len=n)
        pa.cache_keep_path(kc, vc, ks, bt, act, path, acc, new_act, tree_len=n, layout=layout)

    run = step
    if graph:
        saved = [x.clone() for x in (kc, vc, ks, new_act)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for x, y in zip((kc, vc, ks, new_act), saved):
            x.copy_(y)
        run = g.replay
    lengths = list(ctx)
    for it in range(2):
        qkv.copy_(torch.from_numpy(rng.standard_normal(tuple(qkv.shape), dtype=np.float32)))
        c = verify_case(200 + it, B, S1, V, True)
        p.copy_(torch.from_numpy(c["p"])), qd.copy_(torch.from_numpy(c["q"])), u.copy_(torch.from_numpy(c["u"]))
        tok.copy_(torch.from_numpy(c["tok"]))
        before = [x.clone() for x in (kc, vc, ks)]
        snap = [x.clone() for x in before]
        run()
        torch.cuda.synchronize()
        assert ws.error_flags() == 0
        want = H.verify_reference(c["p"], c["q"], c["tok"], par_np, c["u"], n.cpu().numpy())
        for a, b in zip((acc, path, toks), want):
            assert np.array_equal(a.cpu().numpy(), b)
        # an append of the accepted branch alone
        for b in range(B):
            for i in range(int(want[0][b])):
                s = int(want[1][b, i])
                a = lengths[b] + i
                one = torch.tensor([int(bt_np[b, a // 128]) * 128 + a % 128], dtype=torch.int32, **dev)
                t = b * S1 + s
                pa.qkv_norm_rope_append(q[t:t + 1], k[t:t + 1], v[t:t + 1], w, w, cs, pos[t:t + 1],
                                        torch.zeros((1, NQ, 128), dtype=torch.uint8, **dev),
                                        torch.zeros((1, NQ), **dev), before[0], before[1], one, before[2], vs,
                                        tb[t:t + 1], layout=layout)
            lengths[b] += int(want[0][b])
        assert new_act.cpu().tolist() == lengths
        for x, y in zip((kc, vc, ks), before):
            x, y = H.by_position(x, layout), H.by_position(y, layout)
            for b in range(B):
                a = torch.arange(lengths[b], device="cuda")
                ids = bt[b].long()[a // 128]
                assert torch.equal(x[ids, a % 128], y[ids, a % 128])
        # the drafted nodes' attention over the cache as it was before the move
        pa.qkv_norm_rope_append(q, k, v, w, w, cs, pos, qc, qs, *snap[:2], slots, snap[2], vs, tb, layout=layout)
        case = dict(B=B, S1=S1, NQ=NQ, NKV=NKV, layout=layout, n=n, act=act, bt=bt, kc=snap[0], vc=snap[1],
                    ks=snap[2], q=qc, qs=qs, vs=vs, mask=mask)
        check_tree({k_: x.cpu() if isinstance(x, torch.Tensor) else x for k_, x in case.items()}, out)


# ---- sizes and calls at the borders ------------------------------------------------

def test_tree_decode_signs_of_scales():
    """Scales of either sign and a zero one: the maximum is then over S k_scale
    with its sign turned."""
    c = H.tree_case(21, [400, 130], 5, 16, 2, 0)
    c["qs"][::2] *= -1
    c["qs"][1, 3] = 0
    ks = H.by_position(c["ks"], 0)
    ks[:, ::3] *= -1
    check_tree(c, run_tree(c))


@pytest.mark.parametrize("layout", [0, 1])
def test_tree_decode_wide_items_cut_by_runs(layout):
    """Row tiles of 128, 128 and 64 rows (32 in the ragged sequence's last), cut
    by the runs' ends, next to sequences of nothing."""
    c = H.tree_case(22, [6000, 0, 2500, 900], 40, 16, 2, layout, n=[40, 0, 20, 33])
    check_tree(c, run_tree(c))


def test_tree_decode_most_sequences():
    rng = np.random.default_rng(23)
    c = H.tree_case(23, [int(x) for x in rng.integers(0, 140, 1024)], 3, 4, 1, 1,
                    n=[int(x) for x in rng.integers(0, 4, 1024)])
    check_tree(c, run_tree(c))


def test_tree_decode_one_workspace_for_calls_of_several_shapes():
    pa = _pa()
    ws = pa.TreeWorkspace(8, 64, 96, 8)
    for i, (ctx, S1, NQ, NKV) in enumerate([([9000, 300], 8, 96, 8), ([5], 1, 1, 1), ([2000] * 3, 64, 48, 4),
                                            ([0, 1], 4, 4, 4), ([9000, 300], 8, 96, 8)]):
        c = H.tree_case(30 + i, ctx, S1, NQ, NKV, i % 2)
        check_tree(c, run_tree(c, ws=ws))


def test_tree_decode_two_graphs_at_once():
    """Two captured calls with a workspace each, replayed on two streams."""
    pa = _pa()
    runs = []
    for i in range(2):
        c = H.tree_case(40 + i, [5000 + 900 * i, 70], 6, 24, 2, i)
        g = _cuda(c)
        out = torch.zeros((12, 24, H.D), dtype=torch.bfloat16, device="cuda")
        ws, s = pa.TreeWorkspace(2, 6, 24, 2), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call = pa.prepare_tree_decode(g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"],
                                          g["mask"], out, S1=6, tree_len=g["n"], layout=i, workspace=ws)
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        out.fill_(float("nan"))
        runs.append((c, g, out, ws, s, graph))
    torch.cuda.synchronize()
    for _ in range(20):
        for *_, s, graph in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, _, out, ws, *_ in runs:
        assert ws.error_flags() == 0
        check_tree(c, out)


@pytest.mark.parametrize("layout", [0, 1])
def test_cache_past_32_bit_offsets(layout):
    """The step's cache calls on blocks at the end of caches of 5.2 GB."""
    pa = _pa()
    NB, S1, NQ, NKV = 40000, 4, 16, 8
    c = H.tree_case(50 + layout, [200, 126], S1, NQ, NKV, layout)
    small, at = c["kc"].shape[0], NB - c["kc"].shape[0]
    dev = dict(device="cuda")
    sh = H.cache_shape(layout, NB, NKV)
    kc, vc = (torch.zeros(sh + (128,), dtype=torch.uint8, **dev) for _ in range(2))
    ks = torch.zeros(sh, **dev)
    for big, k in ((kc, "kc"), (vc, "vc"), (ks, "ks")):
        big[at:] = c[k].cuda()
    bt = torch.where(c["bt"] >= 0, c["bt"] + at, -1)
    g = _cuda(c)
    out = torch.zeros((2 * S1, NQ, 128), dtype=torch.bfloat16, **dev)
    pa.tree_decode(g["q"], g["qs"], kc, ks, vc, g["vs"], bt.cuda(), g["act"], g["mask"], out, S1=S1,
                   tree_len=g["n"], layout=layout)
    torch.cuda.synchronize()
    check_tree(c, out)
    path = torch.tensor([[0, 2, 3, -1], [0, 3, -1, -1]], dtype=torch.int32)
    acc = torch.tensor([3, 2], dtype=torch.int32)
    new = torch.zeros(2, dtype=torch.int32, **dev)
    pa.cache_keep_path(kc, vc, ks, bt.cuda(), g["act"], path.cuda(), acc.cuda(), new, tree_len=g["n"], layout=layout)
    want = keep_reference(dict(c, path=path, acc=acc, BS=128))
    for big, w in zip((kc, vc, ks), want):
        assert torch.equal(H.by_position(big[at:], layout).cpu(), w)
    assert torch.equal(new.cpu(), want[3])
    # append to the last block's rows
    T = 5
    a = append_case(51, T, NQ, NKV, 128, 64, torch.bfloat16, layout)
    slots = torch.arange(NB * 128 - T, NB * 128, dtype=torch.int64)
    a.update(slots=torch.arange(small * 128 - T, small * 128, dtype=torch.int64), NB=small, BS=128)
    kc[at:], vc[at:], ks[at:] = 0xA5, 0x5A, -7.0
    qc, qs = torch.zeros((T, NQ, 128), dtype=torch.uint8, **dev), torch.zeros((T, NQ), **dev)
    pa.qkv_norm_rope_append(a["q"].cuda(), a["k"].cuda(), a["v"].cuda(), a["qw"].cuda(), a["kw"].cuda(),
                            a["cs"].cuda(), a["pos"].cuda(), qc, qs, kc, vc, slots.cuda(), ks, a["vs"].cuda(),
                            a["tb"].cuda(), eps=1e-5, interleaved=False, layout=layout)
    torch.cuda.synchronize()
    check_append(a, (qc.cpu(), qs.cpu(), kc[at:].cpu(), vc[at:].cpu(), ks[at:].cpu()))
    assert not kc[:at].any() and not vc[:at].any() and not ks[:at].any()


def test_append_of_no_tokens_and_of_many():
    a = append_case(60, 0, 3, 1, 64, 32, torch.bfloat16, 0)
    assert (run_append(a)[2] == 0xA5).all()
    a = append_case(61, 3001, 10, 2, 128, 64, torch.bfloat16, 1)
    check_append(a, run_append(a))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,V", [(76, 260), (77, 260), (153, 515), (305, 512), (700, 131)])
def test_verify_batches_on_fewer_processors_each(B, V, draft):
    check_verify(verify_case(B, B, 5, V, draft))


def test_verify_tokens_do_not_depend_on_the_batch():
    """A sequence's draw is the same alone and among others."""
    c = verify_case(70, 320, 6, 2000, True)
    acc, path, tokens = check_verify(c)
    for b in (0, 150, 319):
        one = {k: v[b:b + 1] for k, v in c.items()}
        for x, y in zip(run_verify(one), (acc, path, tokens)):
            assert np.array_equal(x[0], y[b])


def test_verify_rows_past_32_bit_offsets():
    """2.5e9 probabilities: the last sequences lie past 2^31 elements."""
    pa = _pa()
    B, S1, V = 600, 16, 262144
    dev = dict(device="cuda")
    p = torch.zeros((B, S1, V), **dev)
    hot = [(b * 1009 + 7) % V for b in range(B)]
    p[torch.arange(B, **dev), 3, torch.tensor(hot, **dev)] = 1.0
    p[:, 0, 11] = 1.0
    tok = torch.full((B, S1), 12, dtype=torch.int32, **dev)
    tok[:, 3] = 11
    par = torch.zeros((B, S1), dtype=torch.int32, **dev)
    u = torch.full((B, S1), 0.5, **dev)
    acc, path, toks = (torch.zeros(s, dtype=torch.int32, **dev) for s in ((B,), (B, S1), (B, S1)))
    pa.tree_verify(p, None, tok, par, u, acc, path, toks)
    torch.cuda.synchronize()
    assert (acc == 2).all() and (path[:, :3].cpu() == torch.tensor([0, 3, -1])).all()
    assert (toks[:, 0] == 11).all() and toks[:, 1].cpu().tolist() == hot and (toks[:, 2:] == -1).all()


@pytest.mark.parametrize("what", ["verify", "keep", "append"])
def test_step_calls_on_another_stream_and_replayed(what):
    pa = _pa()
    side = torch.cuda.Stream()
    if what == "verify":
        c = verify_case(80, 6, 7, 900, True)
        t = {k: torch.from_numpy(v).cuda() for k, v in c.items()}
        got = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((6,), (6, 7), (6, 7))]
        call = pa.prepare_tree_verify(t["p"], t["q"], t["tok"], t["par"], t["u"], *got, tree_len=t["n"], stream=side)
        want = [torch.from_numpy(x) for x in H.verify_reference(c["p"], c["q"], c["tok"], c["par"], c["u"], c["n"])]
    elif what == "keep":
        c = keep_case(81, [100, 7, 300], 9, 2, 0)
        t = _cuda(c)
        got = [t["kc"], t["vc"], t["ks"], torch.zeros(3, dtype=torch.int32, device="cuda")]
        call = pa.prepare_cache_keep_path(t["kc"], t["vc"], t["ks"], t["bt"], t["act"], t["path"], t["acc"], got[3],
                                          tree_len=t["n"], layout=0, stream=side)
        want = keep_reference(c)
    else:
        c = append_case(82, 19, 4, 2, 128, 64, torch.float32, 0)
        want = run_append(c)
        t = _cuda(c)
        got = [torch.zeros_like(want[0]).cuda(), torch.zeros_like(want[1]).cuda(), torch.full_like(want[2], 0xA5).cuda(),
               torch.full_like(want[3], 0x5A).cuda(), torch.full_like(want[4], -7.0).cuda()]
        call = pa.prepare_qkv_norm_rope_append(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["cs"], t["pos"], got[0],
                                               got[1], got[2], got[3], t["slots"], got[4], t["vs"], t["tb"], eps=1e-5,
                                               interleaved=False, layout=0, stream=side)
    clean = [x.clone() for x in got]
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(2):
        for x, y in zip(got, clean):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.cpu(), y)


def test_calls_of_no_sequences():
    pa = _pa()
    c = _cuda(H.tree_case(90, [10], 2, 4, 2, 0))
    no = lambda *s, dt=torch.int32: torch.zeros((0,) + s, dtype=dt, device="cuda")  # noqa: E731
    pa.tree_decode(no(4, 128, dt=torch.uint8), no(4, dt=torch.float32), c["kc"], c["ks"], c["vc"],
                   no(2, 128, dt=torch.float32), no(3), no(), no(2, 2, dt=torch.bool),
                   no(4, 128, dt=torch.bfloat16), S1=2, tree_len=no(), layout=0)
    pa.tree_verify(no(2, 9, dt=torch.float32), None, no(2), no(2), no(2, dt=torch.float32), no(), no(2), no(2))
    pa.cache_keep_path(c["kc"], c["vc"], c["ks"], no(3), no(), no(2), no(), no(), layout=0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("draft", [True, False])
def test_verify_ties_and_their_neighbours(draft):
    """u z Q equal to R (not below it: rejected), and one step to either side,
    for the first draft and the same for the second after it."""
    B, S1, V = 9, 3, 8
    p = np.full((B, S1, V), 1 / 16, np.float32)
    q = np.full((B, S1, V), 1 / 16, np.float32)
    p[:, 0, 1], p[:, 0, 2], p[:, 0, 3] = 0.25, 0.3125 if draft else 0.375, 0.5
    q[:, 0, 1], q[:, 0, 2] = 0.5, 0.25
    step = np.float32(2.0 ** -24)
    u = np.full((B, S1), 0.3, np.float32)
    first = 0.5 if draft else 0.25                      # u Q = R, u = R
    u[0, 1], u[1, 1], u[2, 1] = first - step / 2, first, first + step
    u[3:, 1] = 0.9
    c = dict(p=p, q=q if draft else None, tok=np.tile(np.array([0, 1, 2], np.int32), (B, 1)),
             par=np.tile(np.array([-1, 0, 0], np.int32), (B, 1)), u=u, n=np.full(B, S1, np.int32))
    # after the first is rejected: R = 0.0625 and 0.4375 elsewhere, z = 0.5, Q = 0.25;
    # without draft_probs R = 0.375, z = 0.75
    edge = np.float32(0.5)
    for i, x in enumerate((edge - step, edge, edge + step, np.nextafter(edge, np.float32(0)),
                           np.nextafter(edge, np.float32(1)), 0.0)):
        u[3 + i, 2] = x
    got = check_verify(c)[1][:, 1].tolist()
    assert got[0] == 1 and 1 not in got[1:] and [x == 2 for x in got[3:]] == [True, False, False, True, False, True]


@pytest.mark.parametrize("D,rd,inter", [(64, 32, False), (128, 128, True), (256, 64, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rows_at_the_ends_of_the_range(D, rd, inter, norm):
    """Rows whose squares leave the float range on either side, rows of zeros and
    weights of 2^-100 beside ordinary rows of the same call."""
    c = append_case(95 + D, 24, 9, 3, D, rd, torch.float32, 1, wdt=torch.float32)
    for t, f in ((1, 2.0 ** 60), (2, 2.0 ** 100), (3, 2.0 ** 122), (4, 2.0 ** -60), (5, 2.0 ** -100), (6, 0.0),
                 (8, 2.0 ** -20), (9, 2.0 ** 20)):
        c["qkv"][t] *= f
    c["kw"] *= 2.0 ** -100
    eps = 1e-5 if D == 128 else 1e-30
    check_append(c, run_append(c, eps=eps, inter=inter, norm=norm), eps=eps, inter=inter, norm=norm)


def test_append_strides_that_do_not_count():
    """One token and one head: their strides may be anything."""
    pa = _pa()
    a = append_case(97, 1, 1, 1, 128, 64, torch.bfloat16, 0)
    want = run_append(a)
    got = [torch.zeros_like(want[0]).cuda(), torch.zeros_like(want[1]).cuda(), torch.full_like(want[2], 0xA5).cuda(),
           torch.full_like(want[3], 0x5A).cuda(), torch.full_like(want[4], -7.0).cuda()]
    odd = lambda t: t.contiguous().cuda().as_strided((1, 1, 128), (7, 3, 1))  # noqa: E731
    pa.qkv_norm_rope_append(odd(a["q"]), odd(a["k"]), odd(a["v"]), a["qw"].cuda(), a["kw"].cuda(), a["cs"].cuda(),
                            a["pos"].cuda(), got[0], got[1], got[2], got[3], a["slots"].cuda(), got[4], a["vs"].cuda(),
                            a["tb"].cuda(), eps=1e-5, interleaved=False, layout=0)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)


def test_verify_random_numbers_at_the_ends():
    """u[0] at 0 and at the last float below 1 draws the first and the last token
    of any mass, wherever they lie."""
    V = 5003
    p = np.zeros((6, 2, V), np.float32)
    u = np.zeros((6, 2), np.float32)
    u[3:, 0] = np.float32(1) - np.float32(2.0 ** -24)
    spots = [(0, V - 1), (17, 18), (2500, 4999)]
    for b in range(6):
        lo, hi = spots[b % 3]
        p[b, :, lo], p[b, :, hi] = 0.25, 0.75
    c = dict(p=p, q=None, tok=np.full((6, 2), 100, np.int32), par=np.tile(np.array([-1, 0], np.int32), (6, 1)), u=u,
             n=np.full(6, 2, np.int32))
    got = check_verify(c)
    assert got[2][:, 0].tolist() == [s[0] for s in spots] + [s[1] for s in spots]


@pytest.mark.parametrize("D,inter,dtype", [(64, False, torch.float32), (128, False, torch.bfloat16),
                                           (128, True, torch.float32), (256, False, torch.bfloat16)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rows_do_not_depend_on_those_beside_them(D, inter, dtype, norm):
    """Rows of zeros, of 2^-110 and of 2^110 among others: the others come out
    as without them, bit for bit."""
    NQ, NKV, T = 9, 3, 8
    c = append_case(100 + D, T, NQ, NKV, D, 32, dtype, 0, wdt=torch.float32)
    c["slots"] = torch.arange(T, dtype=torch.int32)
    clean = run_append(c, inter=inter, norm=norm)
    heads = c["qkv"].view(T, NQ + 2 * NKV, D)
    same = torch.ones((T, NQ + 2 * NKV), dtype=torch.bool)
    for t, h, f in ((0, 0, 0.0), (1, 4, 2.0 ** -110), (2, NQ - 1, 2.0 ** 110), (3, 2, 0.0), (3, 5, 2.0 ** 110),
                    (4, NQ, 0.0), (5, NQ + 1, 2.0 ** -110), (6, NQ + 2, 2.0 ** 110)):
        heads[t, h] *= f
        same[t, h] = False
    got = run_append(c, inter=inter, norm=norm)
    check_append(c, got, inter=inter, norm=norm)
    q, k = same[:, :NQ], same[:, NQ:NQ + NKV]
    assert torch.equal(got[0][q], clean[0][q]) and torch.equal(got[1][q], clean[1][q])
    for i in (2, 4):
        a, b = (x.reshape((-1,) + x.shape[2:])[:T] for x in (got[i], clean[i]))
        assert torch.equal(a[k], b[k])
    assert torch.equal(got[3], clean[3])


@pytest.mark.parametrize("D,rd,inter,dtype", [(64, 32, False, torch.float32), (128, 64, False, torch.bfloat16),
                                              (128, 128, True, torch.float32), (256, 0, False, torch.bfloat16)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rows_with_infinities_and_nans(D, rd, inter, dtype, norm):
    """A row whose y has a NaN is all NaN, scale too; one whose largest value is
    infinite has that scale, NaN where y is infinite and zeros elsewhere; the
    rows beside them are what they are without them."""
    NQ, NKV, T = 9, 3, 8
    c = append_case(110 + D, T, NQ, NKV, D, rd, dtype, 0, wdt=torch.float32)
    c["slots"] = torch.arange(T, dtype=torch.int32)
    clean = run_append(c, inter=inter, norm=norm)
    inf, nan = float("inf"), float("nan")
    heads = c["qkv"].view(T, NQ + 2 * NKV, D)
    heads[0, 0, 3] = inf
    heads[1, 4, D - 1] = -inf
    heads[2, NQ - 1, ::7] = inf
    heads[3, 2, 5] = nan
    heads[4, 1] = 0                                     # nothing beside it
    heads[4, 1, D - 2] = nan
    heads[5, 5] = 0
    heads[5, 5, 0] = -inf
    heads[6, 3, 1], heads[6, 3, 2] = inf, nan
    heads[1, NQ, 0] = inf                               # keys
    heads[2, NQ + 1, D // 2] = nan
    heads[6, NQ + 2, D - 1] = -inf
    got = run_append(c, inter=inter, norm=norm)
    qc, qs, kc, vc, ks = got
    kc, ks = (x.reshape((-1,) + x.shape[2:])[:T] for x in (kc, ks))
    kc0, ks0 = (clean[i].reshape((-1,) + clean[i].shape[2:])[:T] for i in (2, 4))
    assert torch.equal(vc, clean[3])
    for x, w, code, scale, code0, scale0 in ((c["q"], c["qw"], qc, qs, clean[0], clean[1]),
                                             (c["k"], c["kw"], kc, ks, kc0, ks0)):
        y = H.norm_rope_reference(x, w if norm else None, c["cs"], c["pos"], inter, 1e-5)
        amax = y.abs().amax(-1)                         # (NaN if there is one)
        bad = ~torch.isfinite(amax)
        assert bad.any() and torch.isnan(amax).any() and (norm or torch.isinf(amax).any())
        nan_row, inf_row = torch.isnan(amax), torch.isinf(amax)
        assert torch.equal(code[~bad], code0[~bad]) and torch.equal(scale[~bad], scale0[~bad])
        assert torch.isnan(H.value(code[nan_row])).all() and torch.isnan(scale[nan_row]).all()
        assert (scale[inf_row] == inf).all()
        v = H.value(code[inf_row])
        assert torch.equal(torch.isnan(v), torch.isinf(y[inf_row])) and (v[~torch.isnan(v)] == 0).all()


def test_append_takes_nan_angles_and_infinite_weights_for_what_they_are():
    c = append_case(120, 6, 4, 2, 128, 64, torch.float32, 0, wdt=torch.float32)
    c["slots"] = torch.arange(6, dtype=torch.int32)
    c["pos"] = torch.arange(6, dtype=torch.int32)
    clean = run_append(c)
    c["cs"][2, 7] = float("nan")
    got = run_append(c)
    rows = torch.arange(6) != 2
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][rows], clean[1][rows])
    assert torch.isnan(H.value(got[0][2])).all() and torch.isnan(got[1][2]).all()
    c["cs"][2, 7] = 1.0
    c["qw"][70] = float("inf")                          # a channel that is not rotated
    code, scale = H.value(run_append(c)[0]), run_append(c)[1]
    assert (scale == float("inf")).all() and torch.isnan(code[..., 70]).all()
    assert (code[..., torch.arange(128) != 70] == 0).all()


def test_tree_decode_nans_reach_the_output_of_cut_items():
    """NaN query codes, and NaN key scales over many blocks on end, in items that
    runs' ends cut: rows that meet one are NaN, whatever part it lies in."""
    c = H.tree_case(25, [20000, 300], 5, 24, 2, 0)
    clean = run_tree(c).cpu()
    bad = torch.zeros((10, 24), dtype=torch.bool)
    for t, h in ((0, 0), (2, 13), (4, 23), (5, 0), (7, 12), (9, 5)):
        bad[t, h] = True
    keep = c["q"].clone()
    c["q"][bad] = 0x7F
    out = run_tree(c).cpu()
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])
    c["q"] = keep
    ks = H.by_position(c["ks"], 0)
    ks[c["bt"][0, 40:70].long(), :, 1] = float("nan")        # kv head 1 of the first sequence
    out = run_tree(c).cpu()
    bad[:] = False
    bad[:5, 12:] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_tree_decode_nan_query_scales_give_nan_rows():
    """A row's scale is NaN: so is its output, and no other row's."""
    c = H.tree_case(24, [300, 20000] + [100] * 200, 5, 24, 2, 0)      # items cut by runs' ends and whole ones
    clean = run_tree(c).clone()
    bad = torch.zeros((1010, 24), dtype=torch.bool)
    for t, h in ((0, 0), (2, 13), (4, 23), (5, 0), (7, 12), (9, 5), (100, 3), (500, 20), (807, 7)):
        bad[t, h] = True
    c["qs"][bad] = float("nan")
    out = run_tree(c).cpu()
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean.cpu()[~bad])


@pytest.mark.parametrize("what", ["tree_decode", "decode"])
def test_prepared_calls_own_workspace_on_several_streams(what):
    """A workspace that the call made itself is zeroed before the callable is
    handed out, and its memory stays with streams that still run the call."""
    pa = _pa()
    B, S1, NQ, NKV = 2, 4, 12, 2
    c = H.tree_case(26, [3000, 700], S1, NQ, NKV, 0)
    g = _cuda(c)
    shape = (B * S1, NQ, H.D)
    want = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    base = (g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"])
    if what == "decode":
        size = pa.decode_workspace_size(B, S1, NQ, NKV)
        pa.decode(*base, want, S1=S1, layout=0, workspace=pa.DecodeWorkspace(B, S1, NQ, NKV))
        prepare = lambda out, st: pa.prepare_decode(*base, out, S1=S1, layout=0, stream=st)  # noqa: E731
        direct = lambda out, st: pa.decode(*base, out, S1=S1, layout=0, stream=st)  # noqa: E731
    else:
        size = pa.tree_decode_workspace_size(B, S1, NQ, NKV)
        pa.tree_decode(*base, g["mask"], want, S1=S1, layout=0, workspace=pa.TreeWorkspace(B, S1, NQ, NKV))
        prepare = lambda out, st: pa.prepare_tree_decode(*base, g["mask"], out, S1=S1, layout=0, stream=st)  # noqa: E731
        direct = lambda out, st: pa.tree_decode(*base, g["mask"], out, S1=S1, layout=0, stream=st)  # noqa: E731
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        torch.cuda._sleep(20_000_000)                    # some milliseconds
    call = prepare(outs[0], a)
    assert a.query()                                     # zeroed by now
    with torch.cuda.stream(b):
        torch.cuda._sleep(20_000_000)
    call(stream=b)
    del call
    with torch.cuda.stream(a):                           # what would take the memory over
        junk = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    call = prepare(outs[1], None)
    call()
    b.wait_stream(torch.cuda.current_stream())           # (one workspace: one call after the other)
    call(stream=b)
    direct(outs[2], a)                                   # made and given back on the call's stream
    direct(outs[3], b)
    torch.cuda.synchronize()
    del junk
    for out in outs:
        if what == "decode":
            # which CTA merges a sequence's parts, and so the order of FP32 sums, is not
            # fixed: a few roundings and exponentials (2^-20 of the mass, which is at most
            # max|V| = 448 times the largest scale), then a BF16 rounding either way (2^-7)
            tol = 2.0 ** -7 * want.double().abs() + 2.0 ** -20 * 448 * float(c["vs"].max())
            assert ((out.double() - want.double()).abs() <= tol).all()
        else:
            assert torch.equal(out, want)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("S1,V", [(257, 515), (1024, 2048)])
def test_verify_most_nodes(S1, V, draft):
    """More nodes than a CTA has threads: a node with nearly all others as
    rejected children, the same with repeated tokens, a chain that is accepted to
    its end, random trees, and sequences of no and of one node."""
    c = verify_case(1300 + S1, 7, S1, V, draft, width=6)
    rng = np.random.default_rng(S1)
    c["n"][:] = [S1, S1, S1, S1, 0, 1, S1 - 1]
    for b in (0, 1):
        c["par"][b, 1:] = 0
        c["u"][b, 1:] = np.float32(0.999)
        c["p"][b, 0] = np.float32(1 / V)
        if draft:
            c["q"][b, 0] = 0
            c["q"][b, 0, :V // 2] = np.float32(4 / V)    # p / q = 1 / 4 where drafted from
            c["tok"][b, 1:] = rng.integers(0, V // 2, S1 - 1)
        else:
            c["tok"][b, 1:] = rng.permutation(V)[:S1 - 1] if b == 0 else rng.integers(0, V // 8, S1 - 1)
    c["par"][2, 1:] = np.arange(S1 - 1)
    if draft:
        c["q"][2] = c["p"][2]
        c["u"][2, 1:] = np.minimum(c["u"][2, 1:], np.float32(0.99))
    else:
        c["u"][2, 1:] = 0
    c["tok"][2, 1:] = c["p"][2, :-1].argmax(-1)
    acc, path, tokens = check_verify(c)
    assert acc[0] == 1 and acc[1] == 1 and acc[2] == S1 and acc[4] == 0 and acc[5] == 1
    assert path[2].tolist() == list(range(S1))


def test_tree_decode_scores_past_the_floats_integers():
    """Scores of 1e8 to 1e14, where FP32 steps are larger than the exponents' whole
    range: the largest score's key takes all, equal ones share."""
    c = H.tree_case(27, [700, 5000], 4, 12, 2, 0)
    kc, vc, ks = (H.by_position(c[k], 0) for k in ("kc", "vc", "ks"))
    one = torch.full((), 1.0).to(H.F8).view(torch.uint8)
    c["q"][:] = one
    kc[:] = one                                          # S = 128 everywhere
    keep = ks.clone()
    for f in (1e7, 1e10, 1e13):
        ks[:] = f
        c["qs"][:] = 1.0
        for b, (at, n) in enumerate(((650, 4), (77, 4))):
            ks[c["bt"][b, at // 128].long(), at % 128] = 1.5 * f
        out = run_tree(c).double().cpu()
        for b, at in enumerate((650, 77)):
            want = H.value(vc[c["bt"][b, at // 128].long(), at % 128]) * c["vs"][b].double()   # [NKV, D]
            want = want.repeat_interleave(6, 0)[None].expand(4, 12, 128)
            got = out[4 * b:4 * b + 4]
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all(), f
        # negative scales: all others are far above the one
        c["qs"][:] = -1.0
        assert torch.isfinite(run_tree(c)).all()
    # all equal: the mean of what a row sees
    ks[:] = 1e11
    c["qs"][:] = 1.0
    out = run_tree(c).double().cpu()
    c["ks"] = torch.full_like(keep, 0.01)
    ref, tol = H.tree_reference(c)
    assert ((out - ref).abs() <= tol).all()


@pytest.mark.parametrize("layout", [0, 1])
def test_tree_decode_most_rows(layout):
    """The most drafted tokens and the largest group: 16384 rows a kv head, in
    items that see nothing of one another."""
    c = H.tree_case(28, [100, 0], 128, 128, 1, layout, n=[128, 61])
    check_tree(c, run_tree(c))


@pytest.mark.parametrize("inside", [False, True])
def test_prepared_calls_own_workspace_in_a_graph(inside):
    """Prepared before the capture, or within it: the callable's workspace serves
    every replay."""
    pa = _pa()
    c = H.tree_case(29, [2000, 90], 4, 12, 2, 0)
    want = run_tree(c)
    g = _cuda(c)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    prepare = lambda: pa.prepare_tree_decode(  # noqa: E731
        g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"], g["mask"], out, S1=4, layout=0)
    torch.cuda.synchronize()
    call = None if inside else prepare()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call = prepare() if inside else call
        call(stream=side)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del graph, call
    torch.cuda.synchronize()


def test_tree_decode_nans_in_nodes_that_are_not_seen():
    """K codes and key scales of a drafted node that are NaN or infinite: rows
    whose mask leaves the node out are what they are without it."""
    c = H.tree_case(140, [125, 300, 0], 6, 12, 2, 0)
    c["mask"][:] = torch.from_numpy(H.ancestor_mask([-1, 0, 0, 1, 2, 1]))
    clean = run_tree(c).cpu().view(3, 6, 12, 128)
    kc, ks = H.by_position(c["kc"], 0), H.by_position(c["ks"], 0)
    for b, what in enumerate(("code", "scale", "inf")):
        pos = int(c["act"][b]) - 6 + 2                   # node 2, an ancestor of 2 and 4
        at = int(c["bt"][b, pos // 128]), pos % 128
        if what == "code":
            kc[at] = 0x7F
        else:
            ks[at] = float("nan" if what == "scale" else "inf")
    out = run_tree(c).cpu().view(3, 6, 12, 128)
    rest = [0, 1, 3, 5]
    assert torch.equal(out[:, rest], clean[:, rest])
    assert torch.isnan(out[:2, [2, 4]]).all()


def test_tree_lengths_out_of_range_masks_of_any_byte_and_float8_tensors():
    c = H.tree_case(141, [200, 30, 10, 129], 5, 8, 2, 1)
    c["n"] = torch.tensor([9, -2, 5, 3], dtype=torch.int32)    # clamped to 5 and 0
    c["mask"] = c["mask"].to(torch.uint8) * torch.tensor([1, 2, 128, 255], dtype=torch.uint8)[:, None, None]
    want = run_tree(c)
    check_tree(c, want)
    f = dict(c, **{k: c[k].view(H.F8) for k in ("q", "kc", "vc")})
    assert torch.equal(run_tree(f), want)


def test_verify_and_keep_lengths_out_of_range_and_none():
    c = verify_case(142, 6, 5, 300, True)
    c["n"][:] = [9, -1, 5, 100, 0, 3]
    check_verify(c)
    c = keep_case(143, [100, 250, 7], 12, 2, 1)
    c["n"] = torch.tensor([40, -3, 12], dtype=torch.int32)
    c["act"] += 12
    check_keep(c)
    pa = _pa()
    c["n"][:] = 12
    want = keep_reference(c)
    g = _cuda(c)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    pa.cache_keep_path(g["kc"], g["vc"], g["ks"], g["bt"], g["act"], g["path"], g["acc"], new, layout=1)
    for a, b in zip((g["kc"], g["vc"], g["ks"]), want):
        assert torch.equal(H.by_position(a.cpu(), 1), b)
    assert torch.equal(new.cpu(), want[3])


def test_append_indices_of_both_widths_float8_outputs_and_strides_of_each_input():
    """positions int64 beside slots int32 and the other way round; q, k and v of
    three tensors with strides of their own."""
    pa = _pa()
    for pdt, sdt in ((torch.int64, torch.int32), (torch.int32, torch.int64)):
        c = append_case(144, 23, 5, 2, 128, 64, torch.bfloat16, 0)
        want = run_append(c)
        got = [torch.zeros_like(want[0]).cuda().view(H.F8), torch.zeros_like(want[1]).cuda(),
               torch.full_like(want[2], 0xA5).cuda().view(H.F8), torch.full_like(want[3], 0x5A).cuda().view(H.F8),
               torch.full_like(want[4], -7.0).cuda()]
        wide = lambda t, more: torch.cat([t.flatten(1), t.new_zeros(23, more)], 1).cuda()[:, :t[0].numel()].view(t.shape)  # noqa: E731
        q, k, v = wide(c["q"], 8), c["k"].contiguous().cuda(), wide(c["v"], 4096)
        assert len({q.stride(0), k.stride(0), v.stride(0)}) == 3
        pa.qkv_norm_rope_append(q, k, v, c["qw"].cuda(), c["kw"].cuda(), c["cs"].cuda(), c["pos"].to(pdt).cuda(), got[0],
                                got[1], got[2], got[3], c["slots"].to(sdt).cuda(), got[4], c["vs"].cuda(), c["tb"].cuda(),
                                layout=0)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.cpu().view(y.dtype), y)


def test_append_of_zeros_without_eps_writes_zeros():
    c = append_case(145, 4, 3, 1, 64, 32, torch.float32, 0)
    c["qkv"][1] = 0
    got = run_append(c, eps=0.0)
    assert (got[0][1] == 0).all() and (got[1][1] == 0).all()
    assert torch.isfinite(H.value(got[0])).all() and torch.isfinite(got[1]).all()
