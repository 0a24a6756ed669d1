"""The ragged serving step's operators on the GPU against plain 64-bit forms: the
plan of blocks and slots, the append with several position axes, attention to a
window and the first tokens, log probabilities, and a run of them together."""
import math

import numpy as np
import pytest

from tests import _draft_helpers as H
from tests import _ragged_helpers as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BS, D = R.BS, R.D


def _pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_paged_kv_block_gb300 as pa
    return pa


def _cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- window attention -----------------------------------------------------------------

def window_call(g, out, ws, prepare=False, **kw):
    pa = _pa()
    fn = pa.prepare_window_attention if prepare else pa.window_attention
    args = dict(window=g["window"], sinks=g["sinks"], max_tokens=g.get("max_tokens", g["most"]), layout=g["layout"],
                workspace=ws)
    args.update(kw)
    return fn(g["q"], g["qs"], g["kc"], g["ks"], g["vc"], g["vs"], g["bt"], g["act"], g["cu"], out, **args)


def empty_out(g):
    return torch.full((g["q"].shape[0], g["NQ"], D), math.nan, dtype=torch.bfloat16, device="cuda")


def workspace(g):
    return _pa().WindowWorkspace(g.get("max_tokens", g["most"]), g["NQ"], g["NKV"])


def run_window(c, ws=None, **kw):
    g = _cuda(c)
    out = empty_out(g)
    ws = ws or workspace(g)
    window_call(g, out, ws, **kw)
    torch.cuda.synchronize()
    assert ws.error_flags() == 0
    return out


def check_window(c, out, scale=None):
    ref, tol = R.window_reference(_cuda(c), scale)
    got = out.double()
    behind = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), behind)          # (rows behind the last sequence: as they were)
    bad = ((got - ref).abs() > tol) & ~behind
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() - tol)[~behind].max()),
                           [tuple(int(i) for i in x) for x in bad.nonzero()[:4]])


WINDOWS = [
    # ctx, new, NQ, NKV, layout, window, sinks, rows behind
    ([0], [1], 1, 1, 0, 1, 0, 0),                          # nothing but itself
    ([5, 0, 126], [1, 1, 1], 12, 1, 1, 3, 0, 2),
    ([127, 128, 129, 1000], [1, 1, 1, 1], 16, 4, 0, 128, 0, 0),     # a window of a block
    ([127, 128, 129, 1000], [1, 1, 1, 1], 16, 4, 0, 129, 1, 0),
    ([500, 255, 2000], [1, 1, 1], 96, 8, 1, 64, 5, 0),     # sinks and window apart, and touching
    ([500, 255, 2000], [1, 1, 1], 96, 8, 0, 300, 200, 1),  # sinks of two blocks
    ([700, 3], [1, 1], 8, 2, 0, None, 0, 0),               # no window
    ([700, 3], [1, 1], 8, 2, 0, None, 10, 0),
    ([90], [1], 128, 1, 1, 50, 3, 0),                      # the largest group
    ([400, 20], [3, 2], 12, 1, 0, 100, 2, 0),              # 36 rows
    ([1100, 40, 7], [10, 0, 11], 12, 1, 1, 130, 4, 3),     # around a tile's end, a sequence of no tokens
    ([260, 600], [21, 22], 12, 1, 0, 256, 130, 0),         # around an item's end
    ([0, 0], [300, 129], 4, 2, 1, 100, 8, 0),              # prompts from the begin
    ([0], [700], 12, 2, 0, None, 0, 0),
    ([333, 0, 50, 4], [1, 257, 64, 1], 48, 8, 0, 200, 4, 5),   # decoding and chunks
    ([1500], [130], 15, 3, 1, 1, 0, 0),                    # only itself, a chunk
    ([1500], [130], 15, 3, 1, 1, 300, 0),                  # itself and the sinks
    ([3000], [257], 1, 1, 0, 1000, 64, 0),                 # 257 rows of one head
]


@pytest.mark.parametrize("i", range(len(WINDOWS)))
def test_window_attention_matches_64_bit(i):
    ctx, new, NQ, NKV, layout, window, sinks, behind = WINDOWS[i]
    c = R.window_case(200 + i, ctx, new, NQ, NKV, layout, window, sinks, rows_behind=behind, room=i % 3)
    check_window(c, run_window(c))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_window_attention_long_contexts_are_split_and_joined(layout, new):
    c = R.window_case(7, [20000, 3], [new, 1], 12, 1, layout, None, 0)
    check_window(c, run_window(c))


def test_window_attention_many_sequences():
    rng = np.random.default_rng(3)
    ctx = [int(x) for x in rng.integers(0, 900, 1024)]
    new = [int(x) for x in rng.integers(0, 4, 1024)]
    c = R.window_case(8, ctx, new, 4, 2, 0, 200, 4, rows_behind=7, device="cuda")
    check_window(c, run_window(c))


def test_window_attention_more_items_than_schedule_entries():
    """More than 1024 items a kv head: several share an entry."""
    c = R.window_case(9, [0, 10, 50], [3, 15000, 14000], 12, 1, 1, 8, 2, device="cuda")
    check_window(c, run_window(c))


@pytest.mark.parametrize("most", [1, 3, 40])
def test_window_attention_lengths_out_of_order(most):
    """More tokens than positions, than max_tokens and than rows; lengths past the table,
    and below zero."""
    c = R.window_case(10, [100, 30, 0, 64], [5, 45, 9, 3], 12, 2, 0, 40, 3)
    c["bt"] = torch.where((c["bt"] < 0) | (c["bt"] > 10 ** 5), 1, c["bt"])
    for k in ("kc", "vc", "ks"):                          # (other positions are seen now)
        fresh = R.window_case(10, [100, 30, 0, 64], [5, 45, 9, 3], 12, 2, 0, None, 0)[k]
        n = min(fresh.shape[0], c[k].shape[0])
        c[k][:n] = fresh[:n]
        c[k][(c[k] == R.NAN_CODE) if k != "ks" else c[k].isnan()] = 1
    c["act"] = torch.tensor([105, 20, -4, 10 ** 6], dtype=torch.int32)
    c["cu"][4] = 60
    c["max_tokens"] = most
    check_window(c, run_window(c))


@pytest.mark.parametrize("layout", [0, 1])
def test_window_attention_of_a_mixed_batch_time_after_time(layout):
    """Chunks and single tokens of many lengths, sinks behind most windows: each part of the
    kernel runs ahead of the others now and then."""
    ctx = [1, 1903, 0, 127, 1, 1, 129, 1, 127, 127, 127, 129, 129, 129, 0, 128, 129]
    new = [22, 0, 1, 2, 35, 1, 1, 22, 0, 1, 487, 2, 1, 1, 598, 1, 39]
    c = R.window_case(61, ctx, new, 32, 2, layout, 129, 700)
    first = run_window(c)
    check_window(c, first)
    for _ in range(20):
        assert torch.equal(run_window(c).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("most", [5, 400])
def test_window_attention_refuses_rows_that_decrease(most):
    """A bit of the error word, no more; the next call is not touched by it."""
    c = R.window_case(12, [300, 900, 20], [2, 5, 1], 8, 2, 0, None, 0)
    c["max_tokens"] = most
    g = _cuda(c)
    ws, out = workspace(g), empty_out(g)
    for cu in ([0, 8, 3, 8], [0, 8, 0, 8], [9, 7, 7, 8], [0, -2 ** 31, 2 ** 31 - 1, 0]):
        window_call({**g, "cu": _i32(*cu)}, out, ws)
        assert ws.error_flags() == 16384
        ws.clear_error_flags()
    check_window(c, run_window(c, ws))


def test_window_attention_bad_block_ids_read_block_zero():
    c = R.window_case(11, [300, 200], [2, 1], 8, 2, 0, None, 0)
    c["bt"][0, 1], c["bt"][1, 0] = -3, c["kc"].shape[0]
    for k in ("kc", "vc", "ks"):
        c[k][(c[k] == R.NAN_CODE) if k != "ks" else c[k].isnan()] = 1
    check_window(c, run_window(c))


def test_window_attention_scale_signs_and_extreme_scores():
    c = R.window_case(12, [400, 1000], [20, 1], 12, 2, 0, 150, 20)
    check_window(c, run_window(c, softmax_scale=-0.05), scale=-0.05)
    check_window(c, run_window(c, softmax_scale=0.0), scale=0.0)
    c["qs"][::2] *= -1
    check_window(c, run_window(c))
    c["ks"] *= 40                                          # a few keys take all
    check_window(c, run_window(c))


def test_window_attention_scores_past_the_floats_integers():
    """Scores past 2^22: the largest key takes all."""
    c = R.window_case(13, [500], [30], 4, 1, 1, 200, 3)
    c["ks"] *= 1e7
    out = run_window(c).double().cpu()
    ref, tol = R.window_reference(c)
    # the row's two largest scores are further apart than their roundings
    kc, ks = (H.by_position(c[k], 1) for k in ("kc", "ks"))
    pos = torch.arange(530)
    blk = c["bt"][0].long()[pos // BS]
    ok = (blk >= 0) & (blk < kc.shape[0])
    K = torch.where(ok[:, None], H.value(kc[blk * ok, pos % BS, 0]) * ks[blk * ok, pos % BS, 0].double()[:, None], 0)
    s = torch.einsum("thd,kd->thk", H.value(c["q"]) * c["qs"][..., None].double(), K) * D ** -0.5
    far = torch.arange(500, 530)[:, None] - pos[None]
    s = torch.where(((far >= 0) & ((far < 200) | (pos < 3)))[:, None], s, -math.inf)
    top = s.topk(2, -1).values
    clear = (top[..., 0] - top[..., 1]) > 1000 + top[..., 0].abs() * 2.0 ** -15
    assert clear.sum() > 60
    assert torch.isfinite(out).all()
    lone = (out - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -30
    assert lone[clear].all()


def test_window_attention_nans_reach_the_rows_that_see_them_and_no_others():
    c = R.window_case(14, [300, 5000], [60, 1], 12, 2, 0, 100, 4)
    blk = c["bt"][0].long()
    p = 310                                                # seen by the tokens at 310 .. 409
    c["ks"][blk[p // BS], p % BS, 1] = math.nan
    c["qs"][7, 2] = math.nan
    out = run_window(c).cpu()
    want = torch.zeros((61, 12), dtype=torch.bool)
    want[10:60, 6:] = True                                 # tokens 310 .. 359 of sequence 0, kv head 1
    want[7, 2] = True
    assert torch.equal(out.isnan().any(-1), want) and torch.equal(out.isnan().all(-1), want)


def test_window_attention_nans_reach_the_output_of_cut_items():
    c = R.window_case(15, [20000], [1], 4, 1, 0, None, 0)
    blk = c["bt"][0].long()
    c["ks"][blk[50], :, 0] = math.nan
    assert run_window(c).isnan().all()


def test_window_attention_is_repeatable_bit_for_bit():
    c = R.window_case(16, [5000, 70, 900], [30, 1, 200], 24, 2, 1, 2000, 10)
    ws = workspace(c)
    a = run_window(c, ws)
    for _ in range(3):
        assert torch.equal(run_window(c, ws), a)


def test_window_attention_rows_do_not_depend_on_how_they_come():
    """A prompt in one chunk and token by token: within the roundings of both."""
    c = R.window_case(17, [0], [140], 8, 2, 0, 50, 3, device="cuda")
    whole = run_window(c)
    ref, tol = R.window_reference(c)
    for t in (0, 3, 49, 50, 51, 127, 128, 139):
        one = dict(c, q=c["q"][t:t + 1], qs=c["qs"][t:t + 1], act=_i32(t + 1), cu=_i32(0, 1), most=1)
        got = run_window(one).double()
        assert ((got - ref[t:t + 1]).abs() <= tol[t:t + 1]).all()
        assert ((got - whole[t:t + 1].double()).abs() <= 2 * tol[t:t + 1]).all()


def test_window_attention_of_everything_agrees_with_tree_decode():
    pa = _pa()
    c = _cuda(R.window_case(18, [700, 90], [4, 4], 12, 2, 0, None, 0))
    out = run_window(c)
    other = empty_out(c)
    mask = torch.ones((4, 4), dtype=torch.bool, device="cuda").tril()
    pa.tree_decode(c["q"], c["qs"], c["kc"], c["ks"], c["vc"], c["vs"], c["bt"], c["act"], mask, other, S1=4,
                   layout=0)
    ref, tol = R.window_reference(c)
    assert ((out.double() - other.double()).abs() <= 2 * tol).all()


def test_window_attention_one_workspace_for_calls_of_several_shapes():
    ws = _pa().WindowWorkspace(300, 96, 8)
    for i, (ctx, new, NQ, NKV) in enumerate([([900], [300], 24, 2), ([20000], [1], 12, 1), ([50, 60], [7, 9], 96, 8)]):
        c = R.window_case(20 + i, ctx, new, NQ, NKV, i % 2, 3000, 4)
        check_window(c, run_window(c, ws))


@pytest.mark.parametrize("own", [False, True])
def test_window_attention_on_another_stream_and_replayed_from_a_graph(own):
    c = R.window_case(23, [3100, 90, 0], [2, 50, 30], 12, 1, 0, 700, 4, rows_behind=3)
    g = _cuda(c)
    out, ws = empty_out(g), None if own else workspace(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = window_call(g, out, ws, prepare=True, stream=side)
    call()
    side.synchronize()
    check_window(c, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    # other lengths and tokens than those it was captured with
    d = R.window_case(24, [1000, 2990, 17], [60, 1, 20], 12, 1, 0, 700, 4, rows_behind=4)
    d["max_tokens"] = c["most"]
    d["q"][:], d["qs"][:] = c["q"], c["qs"]
    for k in ("kc", "vc", "ks", "vs"):
        d[k] = c[k]
    d["bt"] = torch.randint(0, c["kc"].shape[0], c["bt"].shape, dtype=torch.int32)
    for k in ("kc", "vc", "ks"):
        d[k] = torch.where(d[k] == R.NAN_CODE if k != "ks" else d[k].isnan(), torch.ones_like(d[k]), d[k])
        g[k].copy_(d[k])
    for k in ("bt", "act", "cu"):
        g[k].copy_(d[k])
    d["act"].clamp_(max=c["bt"].shape[1] * BS)
    for _ in range(2):
        out.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_window(d, out)


def test_window_attention_two_graphs_at_once():
    runs = []
    for i in range(2):
        c = R.window_case(30 + i, [4000, 300], [3, 40], 24, 2, i, 2500, 5)
        g = _cuda(c)
        out, ws, s = empty_out(g), workspace(g), torch.cuda.Stream()
        call = window_call(g, out, ws, prepare=True, stream=s)
        torch.cuda.synchronize()
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        runs.append((c, g, out, ws, s, graph))
    torch.cuda.synchronize()
    for _ in range(5):
        for *_, s, graph in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, _, out, ws, *_ in runs:
        assert ws.error_flags() == 0
        check_window(c, out)


@pytest.mark.parametrize("layout", [0, 1])
def test_window_attention_caches_past_32_bit_offsets(layout):
    """Codes and scales behind 2^32 bytes of a cache."""
    NKV, NB = 8, 34000                                     # 4.46 GB of codes
    c = _cuda(R.window_case(40, [900], [3], 16, NKV, layout, 300, 130))
    n = c["kc"].shape[0]
    big = {}
    for k in ("kc", "vc", "ks"):
        big[k] = torch.empty((NB,) + tuple(c[k].shape[1:]), dtype=c[k].dtype, device="cuda")
        big[k][NB - n:] = c[k]
    bt = torch.where((c["bt"] >= 0) & (c["bt"] < n), c["bt"] + (NB - n), c["bt"])
    d = dict(c, bt=bt, **big)
    out = run_window(d)
    check_window(c, out)


def test_window_attention_of_nothing():
    pa = _pa()
    c = _cuda(R.window_case(41, [40], [2], 8, 2, 0, 10, 0))
    e = dict(c, q=c["q"][:0], qs=c["qs"][:0], cu=_i32(0, 0))
    run_window(e)
    z = dict(c, q=c["q"][:0], qs=c["qs"][:0], cu=_i32(0), act=c["act"][:0], bt=c["bt"][:0], vs=c["vs"][:0], B=0)
    window_call(z, empty_out(z), None)
    out = empty_out(c)
    window_call(dict(c, cu=_i32(0, 0)), out, pa.WindowWorkspace(2, 8, 2))
    assert out.isnan().all()                               # (no sequence's rows)


# ---- the plan ---------------------------------------------------------------------------

def run_plan(act, new, pool, head, bt, T, NB, bs=128, slot64=False, call=None):
    pa = _pa()
    B = len(act)
    bt = torch.tensor(bt, dtype=torch.int32, device="cuda").reshape(B, -1)
    slots = torch.full((T,), 77, dtype=torch.int64 if slot64 else torch.int32, device="cuda")
    pos, tb, cu, nact, nhead = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (T, T, B + 1, B, 1))
    pa.plan_batch(_i32(*act), _i32(*new), _i32(*pool), _i32(head), bt, slots, pos, tb, cu, nact, nhead, num_blocks=NB,
                  block_size=bs)
    return [x.cpu().numpy() for x in (bt, slots, pos, tb, cu, nact, nhead)]


def check_plan(act, new, pool, head, bt, T, NB, bs=128, slot64=False):
    got = run_plan(act, new, pool, head, bt, T, NB, bs, slot64)
    want = R.plan_reference(act, new, pool, head, bt, T, NB, bs)
    for name, g, w in zip("table slots positions batch cu lengths head".split(), got, want):
        assert np.array_equal(g, w), name
    return got


def plan_inputs(seed, B, bs, most, reach, pool=None):
    rng = np.random.default_rng(seed)
    act = rng.integers(0, reach, B)
    new = np.where(rng.random(B) < 0.6, 1, rng.integers(0, most + 1, B))
    W = -(-(reach + most) // bs) + 1
    held = -(-act // bs)
    fresh = -(-(act + new) // bs) - held
    NB = int(held.sum() + fresh.sum()) + 11
    ids = rng.permutation(NB)
    bt = np.full((B, W), -1)
    at = 0
    for b in range(B):
        bt[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    left = ids[at:]
    return act, new, left if pool is None else left[:pool], bt, NB


@pytest.mark.parametrize("B,bs,most,reach,slot64", [
    (1, 128, 1, 1, False), (3, 128, 5, 300, True), (64, 128, 1, 9000, False), (200, 16, 700, 2000, True),
    (511, 128, 40, 500, False), (513, 1, 20, 30, True), (1024, 128, 300, 5000, False)])
def test_plan_matches_the_definition(B, bs, most, reach, slot64):
    act, new, pool, bt, NB = plan_inputs(B, B, bs, most, reach)
    T = int(new.sum())
    for head, rows in ((0, T), (3, T + 5), (0, T + 3000)):
        check_plan(act, new, pool, head, bt, rows, NB, bs, slot64)


def test_plan_refusals_of_requests():
    """A pool that runs out, rows that run out, requests longer than their row of the
    table: the others are granted."""
    act, new, pool, bt, NB = plan_inputs(5, 40, 16, 90, 400, pool=30)
    T = int(new.sum())
    for head, rows in ((0, T), (7, T // 2), (29, T), (30, T), (1000, T), (-5, T)):
        check_plan(act, new, pool, head, bt, rows, NB, 16)
    got = check_plan([16, 10, 16, 3], [1, 5, 1, 2], [9, 8], 1, [[1, -1], [2, -1], [3, -1], [4, -1]], 9, 10, 16)
    # the first takes the last block, the second needs none, the third is refused
    assert got[5].tolist() == [17, 15, 16, 5] and got[6].tolist() == [2]
    check_plan([40, 0, 32], [1, 33, 0], [5, 6, 7, 8], 0, [[1, 2], [-1, -1], [3, 4]], 40, 9, 16)


def test_plan_bad_lengths_and_ids():
    big = 2 ** 31 - 1
    check_plan([-3, 5, 20], [2, -1, 4], [3, 99, -2], 0, [[-1, -1], [0, -1], [1, 7]], 8, 8, 16)
    check_plan([big, 0, 7], [big, big, 2], [3, 4], 0, [[0, 1], [-1, -1], [2, 5]], 6, 8, 16)
    check_plan([1] * 1024, [big] * 1024, [3, 4], 0, [[0]] * 1024, 50, 8, 16)


def test_plan_of_nothing():
    pa = _pa()
    check_plan([5, 6], [0, 0], [3], 0, [[1], [2]], 0, 8, 16)
    check_plan([5, 6], [0, 0], [], 0, [[1], [2]], 4, 8, 16)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    cu, head, slots = _i32(9), _i32(9), _i32(5, 5, 5)
    pa.plan_batch(e, e, e, _i32(0), e.reshape(0, 4), slots, _i32(5, 5, 5), _i32(5, 5, 5), cu, e, head, num_blocks=3)
    assert cu.tolist() == [0] and head.tolist() == [0] and slots.tolist() == [-1, -1, -1]


# ---- the append with several axes -------------------------------------------------------

def run_mrope(q, k, v, qw, kw, cs, pos, slots, vs, tb, NB, axis, layout, inter, prepare=False, codes=torch.uint8):
    pa = _pa()
    T, NQ, D_ = q.shape
    NKV = k.shape[1]
    sh = H.cache_shape(layout, NB, NKV)
    qc = torch.full((T, NQ, D_), 0x33, dtype=torch.uint8, device="cuda").view(codes)
    qs = torch.full((T, NQ), 5.0, device="cuda")
    kc, vc = (torch.full(sh + (D_,), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks = torch.full(sh, 5.0, device="cuda")
    args = [x.cuda() if isinstance(x, torch.Tensor) and not x.is_cuda else x for x in
            (q, k, v, qw, kw, cs, pos, qc, qs, kc, vc, slots, ks, vs, tb)]
    if prepare:
        pa.prepare_qkv_norm_mrope_append(*args, pair_axis=axis, interleaved=inter, layout=layout)()
    else:
        pa.qkv_norm_mrope_append(*args, pair_axis=axis, interleaved=inter, layout=layout)
    torch.cuda.synchronize()
    return qc.view(torch.uint8), qs, kc, vc, ks


def mrope_angles(cs, pos, axis):
    """Each token's own row of angles: [T, rotary_dim]."""
    half = cs.shape[1] // 2
    rows = pos.long().clamp(0, cs.shape[0] - 1)[list(axis)].T            # [T, pairs]
    i = torch.arange(half)
    return torch.cat([cs[rows, i], cs[rows, half + i]], 1)


MROPES = [
    # T, NQ, NKV, D, rotary, axes, order, interleaved, dtype, layout, int64 positions
    (1, 8, 2, 128, 128, 3, "sections", False, torch.bfloat16, 0, False),
    (37, 12, 2, 128, 64, 3, "turns", True, torch.float32, 1, True),
    (130, 96, 8, 128, 128, 3, "sections", False, torch.bfloat16, 0, True),
    (64, 5, 3, 64, 32, 2, "turns", False, torch.float32, 0, False),
    (33, 7, 1, 256, 256, 4, "any", True, torch.bfloat16, 1, False),
    (50, 4, 4, 256, 128, 4, "any", False, torch.float32, 1, True),
    (9, 3, 1, 64, 8, 4, "any", True, torch.bfloat16, 0, False),
    (20, 16, 4, 128, 16, 1, "any", False, torch.bfloat16, 0, False),
]


def mrope_case(i):
    T, NQ, NKV, D_, rd, A, order, inter, dt, layout, p64 = MROPES[i]
    rng = np.random.default_rng(500 + i)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    half = rd // 2
    axis = {"sections": [min(A - 1, j * A // half) for j in range(half)], "turns": [j % A for j in range(half)],
            "any": [int(x) for x in rng.integers(0, A, half)]}[order]
    ang = f(500, half) * 9
    qkv = f(T, NQ + 2 * NKV, D_).to(dt)
    NB = T // BS + 2
    slots = torch.from_numpy(rng.permutation(NB * BS)[:T].astype(np.int32))
    slots[::7] = -1
    pos = torch.from_numpy(rng.integers(-3, 510, (A, T + 5)).astype(np.int64 if p64 else np.int32))
    return dict(q=qkv[:, :NQ], k=qkv[:, NQ:NQ + NKV], v=qkv[:, NQ + NKV:], qw=f(D_).to(dt), kw=f(D_).to(dt),
                cs=torch.cat([ang.cos(), ang.sin()], 1), pos=pos, slots=slots,
                vs=torch.from_numpy(rng.uniform(0.005, 0.02, (3, NKV, D_)).astype(np.float32)),
                tb=torch.from_numpy(rng.integers(0, 3, T).astype(np.int32)), NB=NB, axis=axis, layout=layout,
                inter=inter)


@pytest.mark.parametrize("i", range(len(MROPES)))
def test_mrope_append_matches_64_bit(i):
    """Codes: half a step of E4M3 (2^-4 of the value, 2^-10 below the normal range) and
    the FP32 arithmetic before it, 2^-18 of the largest; the scales' 2^-20."""
    c = mrope_case(i)
    T = c["q"].shape[0]
    d = dict(c, pos=c["pos"].cuda()[:, :T])                # (axes further apart than the tokens)
    qc, qs, kc, vc, ks = run_mrope(**d, prepare=i % 2 == 1)
    pos = c["pos"][:, :T]
    # a row of angles a token: the plain rotation of position t
    own = mrope_angles(c["cs"], pos, c["axis"])
    at = torch.arange(T)
    for x, w, codes, scale in ((c["q"], c["qw"], qc.cpu(), qs.cpu()), (c["k"], c["kw"], None, None)):
        y = H.norm_rope_reference(x, w, own, at, c["inter"], 1e-5)
        if codes is None:
            ok = c["slots"] >= 0
            s = c["slots"][ok].long()
            y = y[ok]
            codes = H.by_position(kc.cpu(), c["layout"])[s // BS, s % BS]
            scale = H.by_position(ks.cpu(), c["layout"])[s // BS, s % BS]
        want = y.abs().amax(-1) / 448
        assert ((scale.double() - want).abs() <= 2.0 ** -20 * want).all()
        back = H.value(codes) * scale[..., None].double()
        tol = 2.0 ** -4 * y.abs() + (2.0 ** -10 + 448 * 2.0 ** -18) * scale[..., None].double()
        assert ((back - y).abs() <= tol).all()


@pytest.mark.parametrize("i", range(len(MROPES)))
def test_mrope_append_of_equal_positions_is_the_append(i):
    """Bit for bit, whatever the axes."""
    pa = _pa()
    c = mrope_case(i)
    T, NQ, D_ = c["q"].shape
    same = c["pos"][0, :T].clone()
    c["pos"] = same[None].expand(c["pos"].shape[0], T).contiguous()
    got = run_mrope(**c)
    layout = c["layout"]
    sh = H.cache_shape(layout, c["NB"], c["k"].shape[1])
    qc = torch.full((T, NQ, D_), 0x33, dtype=torch.uint8, device="cuda")
    kc, vc = (torch.full(sh + (D_,), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2))
    qs, ks = torch.full((T, NQ), 5.0, device="cuda"), torch.full(sh, 5.0, device="cuda")
    g = _cuda(c)
    pa.qkv_norm_rope_append(g["q"], g["k"], g["v"], g["qw"], g["kw"], g["cs"], same.cuda(), qc, qs, kc, vc, g["slots"],
                            ks, g["vs"], g["tb"], interleaved=c["inter"], layout=layout)
    for a, b in zip(got, (qc, qs, kc, vc, ks)):
        assert torch.equal(a, b)


# ---- log probabilities ------------------------------------------------------------------

def run_logprobs(x, tok, k, prepare=False, stream=None):
    pa = _pa()
    n = x.shape[0]
    lp, ent = (torch.full((n,), 7.0, device="cuda") for _ in range(2))
    rank = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    ids = torch.full((n, k), 77, dtype=torch.int32, device="cuda") if k else None
    tlp = torch.full((n, k), 7.0, device="cuda") if k else None
    fn = pa.prepare_token_logprobs if prepare else pa.token_logprobs
    call = fn(x, tok, lp, ranks=rank, entropy=ent, top_ids=ids, top_logprobs=tlp, stream=stream)
    if prepare:
        call()
    torch.cuda.synchronize()
    return lp, rank, ent, ids, tlp


def check_logprobs(x, tok, k, got=None, rows=None):
    """FP32: an exponential is off by 2^-21 and by 2^-23 of its exponent, which is below
    32 where it counts (2^-18), a sum of up to 256 of them a thread by 2^-16, the joins
    of 2^12 threads' by 2^-19: together less than 2^-15 of L (no term is negative), which
    is log L's error, beside a few 2^-24 of the result and of the difference x - M. The
    entropy has that on both its parts, the second of which, the sum of |x - M| w / L, is
    at most log V + 1."""
    got = got or run_logprobs(x, tok, k)
    lp, rank, ent, ids, tlp = R.logprob_reference(x, tok, max(k, 1))
    off = 2.0 ** -14
    close = lambda a, b, t: torch.equal(a.isinf(), b.isinf()) and torch.equal(a.isnan(), b.isnan()) and bool(  # noqa: E731
        ((a.double() - b).abs()[b.isfinite()] <= t + 2.0 ** -22 * b.abs()[b.isfinite()]).all())
    assert close(got[0], lp, off)
    assert torch.equal(got[1].long(), rank.long())
    assert close(got[2], ent, off * (math.log(x.shape[1]) + 3))
    if k:
        assert torch.equal(got[3].long(), ids)
        assert close(got[4], tlp, off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V,k,pad", [
    (1, 1, 1, 0), (3, 2, 2, 1), (5, 31, 31, 0), (2, 1000, 32, 7), (1, 8191, 5, 0), (2, 8192, 20, 0),
    (3, 8193, 1, 3), (1, 32003, 5, 0), (4, 65537, 20, 0), (1, 262145, 32, 0), (300, 3001, 7, 5), (700, 50, 0, 0),
    (40, 131072, 0, 0), (160, 20000, 20, 13)])
def test_logprobs_match_64_bit(rows, V, k, pad, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 7 + V)
    x = (4 * torch.randn((rows, V + pad), generator=g, device="cuda")).to(dtype)[:, :V]
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    check_logprobs(x, tok, k)
    # one value at an offset from its elements' 16 bytes, 64-bit tokens, a prepared call
    y = torch.empty(rows * V + 9, dtype=dtype, device="cuda")[3:3 + rows * V].view(rows, V)
    y.copy_(x)
    check_logprobs(y, tok.long(), k, run_logprobs(y, tok.long(), k, prepare=True))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "masked", "few", "two values", "blocks", "zeros", "far"])
def test_logprobs_orders_and_ties(kind, dtype):
    """Ties go to the lowest index, in whatever order the values come."""
    V, k = 70001, 32
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    x = {"equal": torch.full_like(i, 2.5), "rising": i / 8192, "falling": -i / 8192,
         "masked": torch.full_like(i, -math.inf),
         "few": torch.where(i % 20000 == 123, 1.0, -math.inf),
         "two values": torch.where((i * 7919) % 11 < 3, 1.0, 0.0),
         "blocks": torch.where((i > 30000) & (i < 30600), 3 + (i * 31) % 17, (i * 7919) % 5),
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0),
         "far": torch.where(i == 4321, 1e38, -1e38)}[kind][None].to(dtype)
    tok = _i32(4321)
    check_logprobs(x, tok, k)
    check_logprobs(x.expand(3, V).contiguous(), tok.expand(3).contiguous(), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 9001, 70001])
def test_logprobs_ranks_beside_zeros_and_the_largest_values(V, dtype):
    """Zeros of either sign are equal; differences may leave the range of the type."""
    i = torch.arange(V, device="cuda")
    big = torch.finfo(dtype).max
    zeros = torch.where(i % 3 == 0, 1.0, torch.where(i % 2 == 0, 0.0, -0.0))
    ends = torch.where(i % 5 == 0, big, torch.where(i % 5 == 1, -big, torch.where(i % 5 == 2, -math.inf, i.float() / V)))
    x = torch.stack([zeros, zeros, ends, ends, ends, ends]).to(dtype)
    tok = _i32(1, 4, 5, 6, 7, 8)             # -0, 0, the largest, the least, -inf, one between
    *_, rank, _, ids, _ = (None, *run_logprobs(x, tok, 20))
    want = (x.double() > x.double().gather(1, tok.long()[:, None])).sum(-1)
    assert torch.equal(rank.long(), want)
    assert torch.equal(ids.long(), torch.argsort(x.double(), dim=-1, descending=True, stable=True)[:, :20])


def test_logprobs_of_bad_rows_and_tokens():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((7, 9000), generator=g, device="cuda")
    clean = x.clone()
    x[1, 8999], x[3, 5], x[4, 100] = math.nan, math.inf, -math.nan
    x[4, 101:9000] = -math.inf
    x[5, :] = math.nan
    tok = torch.tensor([3, 4, -1, 6, 100, 8, 9000], dtype=torch.int64, device="cuda")
    lp, rank, ent, ids, tlp = run_logprobs(x, tok, 5)
    bad = torch.tensor([0, 1, 0, 1, 1, 1, 0], dtype=torch.bool, device="cuda")
    assert torch.equal(ent.isnan(), bad) and torch.equal(tlp.isnan().all(-1), bad)
    assert torch.equal((ids == -1).all(-1), bad) and (rank[bad] == -1).all()
    assert torch.equal(lp.isnan(), bad | (tok < 0) | (tok >= 9000))
    rows = [0, 2, 6]
    check_logprobs(clean[rows], tok[rows], 5, tuple(t[rows] for t in (lp, rank, ent, ids, tlp)))


def test_logprobs_rows_do_not_depend_on_the_batch():
    """On one and on eight CTAs a row: alternatives and ranks are the same, the sums
    within their roundings."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((400, 40000), generator=g, device="cuda").bfloat16()
    tok = torch.randint(0, 40000, (400,), generator=g, device="cuda", dtype=torch.int32)
    many = run_logprobs(x, tok, 20)
    one = run_logprobs(x[11:12], tok[11:12], 20)
    assert torch.equal(many[1][11:12], one[1]) and torch.equal(many[3][11:12], one[3])
    for a, b in zip(many, one):
        assert ((a[11:12].double() - b.double()).abs() <= 2.0 ** -13 * (1 + b.double().abs())).all()


def test_logprobs_rows_past_32_bit_offsets():
    V = 50001
    x = torch.zeros((2 ** 32 // (2 * V) + 3, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x[-2:] = torch.randn((2, V), generator=g, device="cuda").bfloat16()
    tok = torch.full((x.shape[0],), 40000, dtype=torch.int32, device="cuda")
    got = run_logprobs(x, tok, 3)
    check_logprobs(x[-2:], tok[-2:], 3, tuple(t[-2:] for t in got))


def test_logprobs_on_another_stream_and_replayed():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((6, 30000), generator=g, device="cuda")
    tok = torch.randint(0, 30000, (6,), generator=g, device="cuda")
    pa = _pa()
    lp, ids, tlp = torch.zeros(6, device="cuda"), torch.zeros((6, 4), dtype=torch.int32, device="cuda"), \
        torch.zeros((6, 4), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = pa.prepare_token_logprobs(x, tok, lp, top_ids=ids, top_logprobs=tlp, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(2):
        x.copy_(torch.randn((6, 30000), generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = R.logprob_reference(x, tok, 4)
        assert ((lp.double() - want[0]).abs() <= 2.0 ** -13).all() and torch.equal(ids.long(), want[3])


# ---- a step of all four -----------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
def test_ragged_step(layout, graph):
    """Three steps of five requests, prompts' chunks and single tokens in a padded batch:
    plan, append, attention, log probabilities; against the attention over what the
    caches hold, and the caches against what was appended."""
    pa = _pa()
    rng = np.random.default_rng(60 + layout)
    B, T, NQ, NKV, V, NB, W = 5, 160, 12, 2, 999, 40, 6
    window, sinks, rd = 100, 4, 64
    axis = [0] * 8 + [1] * 12 + [2] * 12
    f = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    w_qkv, w_out = f(64, (NQ + 2 * NKV) * D) / 8, f(NQ * D, V) / 30
    ang = f(400, rd // 2) * 5
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    weight = 1 + f(D) / 8
    act, new_act, lens, head, new_head = z(B), z(B), z(B), z(1), z(1)
    bt = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    pool = torch.from_numpy(rng.permutation(NB).astype(np.int32)).cuda()
    slots, pos, tb, cu = z(T), z(T), z(T), z(B + 1)
    axes = z(3, T)
    x, tok = z(T, 64, dt=torch.float32), z(T)
    qkv = z(T, (NQ + 2 * NKV) * D, dt=torch.float32)
    sh = H.cache_shape(layout, NB, NKV)
    kc, vc = z(*sh, D, dt=torch.uint8), z(*sh, D, dt=torch.uint8)
    ks, vs = z(*sh, dt=torch.float32), torch.full((B, NKV, D), 0.02, device="cuda")
    qc, qs = z(T, NQ, D, dt=torch.uint8), z(T, NQ, dt=torch.float32)
    out, logits = z(T, NQ, D, dt=torch.bfloat16), z(T, V, dt=torch.float32)
    lp, ent, ids, tlp = z(T, dt=torch.float32), z(T, dt=torch.float32), z(T, 3), z(T, 3, dt=torch.float32)
    ws = pa.WindowWorkspace(T, NQ, NKV)

    def step():
        pa.plan_batch(act, lens, pool, head, bt, slots, pos, tb, cu, new_act, new_head, num_blocks=NB)
        # text: all axes one, but for a shift of two that images leave behind
        axes.copy_(torch.stack([pos, pos + 1, pos + 2]))
        torch.matmul(x, w_qkv, out=qkv)
        r = qkv.view(T, NQ + 2 * NKV, D)
        pa.qkv_norm_mrope_append(r[:, :NQ], r[:, NQ:NQ + NKV], r[:, NQ + NKV:], weight, weight, cs, axes, qc, qs, kc, vc,
                                 slots, ks, vs, tb, pair_axis=axis, layout=layout)
        pa.window_attention(qc, qs, kc, ks, vc, vs, bt, new_act, cu, out, window=window, sinks=sinks, layout=layout,
                            workspace=ws)
        torch.matmul(out.float().view(T, -1), w_out, out=logits)
        pa.token_logprobs(logits, tok, lp, entropy=ent, top_ids=ids, top_logprobs=tlp)

    call = step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                         # (of no tokens)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        call = g.replay
    history = [[] for _ in range(B)]
    for new in ([130, 1, 7, 0, 20], [1, 90, 1, 60, 1], [1, 1, 100, 1, 1]):
        before = bt.clone()
        lens.copy_(_i32(*new))
        x.copy_(f(T, 64))
        tok.copy_(torch.from_numpy(rng.integers(0, V, T).astype(np.int32)))
        out.fill_(math.nan)
        call()
        torch.cuda.synchronize()
        assert ws.error_flags() == 0
        n = sum(new)
        plan = R.plan_reference(act.cpu().numpy(), new, pool.cpu().numpy(), int(head), before.cpu().numpy(), T, NB, BS)
        for a, b in zip((bt, slots, pos, tb, cu, new_act, new_head), plan):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))
        # what was appended is in the caches, all steps' of it
        rows = qkv.view(T, NQ + 2 * NKV, D).cpu()
        y = H.norm_rope_reference(rows[:, NQ:NQ + NKV], weight.cpu(), mrope_angles(cs.cpu(), axes.cpu(), axis),
                                  torch.arange(T), False, 1e-5)
        for b in range(B):
            history[b] += [y[t] for t in range(plan[4][b], plan[4][b + 1])]
            p = torch.arange(len(history[b]))
            assert len(p) == int(new_act[b])
            if len(p) == 0:
                continue
            blk = bt[b].cpu().long()[p // BS]
            scale = H.by_position(ks.cpu(), layout)[blk, p % BS].double()[..., None]
            back = H.value(H.by_position(kc.cpu(), layout)[blk, p % BS]) * scale
            want = torch.stack(history[b])
            assert ((back - want).abs() <= 2.0 ** -4 * want.abs() + (2.0 ** -10 + 448 * 2.0 ** -18) * scale).all()
        c = dict(B=B, NQ=NQ, NKV=NKV, layout=layout, window=window, sinks=sinks, act=new_act, bt=bt, cu=cu, kc=kc, vc=vc,
                 ks=ks, q=qc, qs=qs, vs=vs)
        check_window(c, out)
        check_logprobs(logits[:n], tok[:n], 3, (lp[:n], R.logprob_reference(logits[:n], tok[:n], 1)[1], ent[:n], ids[:n],
                                                tlp[:n]))
        act.copy_(new_act)
        head.copy_(new_head)


# ---- empty tensors, slices of others ------------------------------------------------------

def test_empty_slices_of_other_tensors():
    """A used-up pool that begins where the block table does, and alternatives of width 0
    cut from the log probabilities: neither has an element to overlap with."""
    pa = _pa()
    bt = _i32(2, -1, 3, -1).reshape(2, 2)
    slots, pos, tb, cu, nact, nhead = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (2, 2, 2, 3, 2, 1))
    pa.plan_batch(_i32(5, 127), _i32(1, 1), bt.view(-1)[:0], _i32(0), bt, slots, pos, tb, cu, nact, nhead, num_blocks=9)
    assert slots.tolist() == [2 * 128 + 5, 3 * 128 + 127] and nact.tolist() == [6, 128] and nhead.tolist() == [0]
    x, tok = torch.randn((3, 500), device="cuda"), _i32(1, 2, 3)
    lp, ids = torch.empty(3, device="cuda"), torch.empty((3, 4), dtype=torch.int32, device="cuda")
    pa.token_logprobs(x, tok, lp, ranks=ids.view(-1)[:3], top_ids=ids[:, :0], top_logprobs=lp.view(3, 1)[:, :0])
    want = R.logprob_reference(x, tok, 1)
    assert ((lp.double() - want[0]).abs() <= 2.0 ** -14).all() and torch.equal(ids.view(-1)[:3].long(), want[1].long())


# ---- rows that see nothing ------------------------------------------------------------

@pytest.mark.parametrize("most", [2000, 300, 2])
def test_window_attention_rows_that_see_nothing_are_zeros_among_others(most):
    """Refused chunks (their tokens are rows, their lengths as before), positions below
    zero, and tokens behind max_tokens, between and behind sequences that are served."""
    ctx, new = [0, 0, 900, 0, 40, 0, 3, 0, 0], [700, 1, 3, 0, 400, 1, 2, 2000, 55]
    c = R.window_case(62, ctx, new, 12, 2, 0, 200, 4, rows_behind=9, device="cuda")
    c["act"] = torch.tensor([0, 1, 903, 0, 250, 1, 5, 0, 20], dtype=torch.int32, device="cuda")
    c["bt"] = torch.where((c["bt"] < 0) | (c["bt"] > 10 ** 5), 1, c["bt"])
    for k in ("kc", "vc", "ks"):                          # (other positions are seen now)
        c[k][(c[k] == R.NAN_CODE) if k != "ks" else c[k].isnan()] = 1
    c["max_tokens"] = most
    check_window(c, run_window(c))


def test_window_attention_a_refused_chunk_does_not_hold_up_the_others():
    """The zeros of 5000 rows of a refused prompt beside 32 decoding requests (123 MB) are
    spread over the GPU: at most five times what writing them alone takes."""
    c = R.window_case(63, [1000] * 33, [1] * 32 + [5000], 96, 8, 0, 500, 4, device="cuda")
    c["act"][32] = 0
    alone = dict(c, cu=c["cu"].clone())
    alone["cu"][33] = 32
    ws, out = workspace(c), empty_out(c)

    def best(call):
        t = []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(200000)                      # (the launches are all enqueued by then)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
        return min(t[2:])
    with_it, without = (best(window_call(d, out, ws, prepare=True)) for d in (c, alone))
    zeros = best(lambda: out[32:].zero_())
    print("with %.4f without %.4f zeros %.4f ms" % (with_it, without, zeros))
    out.fill_(math.nan)
    window_call(c, out, ws)
    torch.cuda.synchronize()
    assert not out[32:].any() and not out.isnan().any() and ws.error_flags() == 0
    assert with_it - without <= 5 * zeros, (with_it, without, zeros)


# ---- log probabilities far from zero --------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rise", [0, 5, 9])
@pytest.mark.parametrize("base", [30, 1000, -900, 1023, -1026, 5000, -70000])
@pytest.mark.parametrize("masked", [False, True])
def test_logprobs_of_one_thread_far_from_zero(base, rise, dtype, masked):
    """A row's weight in the values of one thread, so that what its reference's rounding
    is off by (up to 2^-14 of the exponent at 1000) is not averaged over threads. Two
    groups of 16 values, the second higher by `rise`: less and more than what makes a
    thread take another reference.

    FP32: an exponential is off by 2^-22 and by 2^-24 of its exponent (times ln 2), which
    is below 2^5 where it counts (2^-19.5); its thread's sum has 18 roundings (2^-19.8);
    the joins change nothing, all other threads' sums are 0 beside it. Together 2^-18 of
    L, which is log L's error; the logarithm's and the differences' are 2^-22 of them.
    Entropy: the same weights are in s and L, so that their errors count times the mean
    distance of x from its mean, below 4, and s has roundings of its own, 2^-19.5 of its
    terms' magnitudes, below 8 L."""
    V, rows, off = 16384, 320, 2.0 ** -18
    piece = 4 if dtype == torch.float32 else 8             # values; a thread's next is 512 pieces further
    g = torch.Generator(device="cuda")
    g.manual_seed(abs(base) + rise)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = torch.full((rows, V), base - 400.0, device="cuda").add_(rnd(rows, V))
    thread = torch.randint(0, 512, (rows, 1, 1), generator=g, device="cuda")
    at = torch.arange(32 // piece, device="cuda")[None, :, None] * 512 * piece + thread * piece
    at = (at + torch.arange(piece, device="cuda")).flatten(1)
    high = base + 2 * rnd(rows, 32)
    high[:, 16:] += rise
    x.scatter_(1, at, high)
    if masked:
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.3] = -math.inf
    x = x.to(dtype)
    tok = at[torch.arange(rows, device="cuda"), torch.randint(0, 32, (rows,), generator=g, device="cuda")].int()
    got = run_logprobs(x, tok, 5)
    lp, rank, ent, ids, tlp = R.logprob_reference(x, tok, 5)
    for a, b, t in ((got[0], lp, off), (got[4], tlp, off), (got[2], ent, 5 * off + 8 * 2.0 ** -19.5)):
        assert torch.equal(a.isinf(), b.isinf()) and torch.equal(a.isnan(), b.isnan())
        fin = b.isfinite()
        err = (a.double() - b).abs()[fin] - 2.0 ** -22 * b.abs()[fin]
        assert err.max() <= t, (float(err.max()), t)
    assert torch.equal(got[1].long(), rank.long()) and torch.equal(got[3].long(), ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V,lo,hi", [(400, 40000, 1000, 1060), (3, 40000, -1060, -1000), (400, 9001, 900, 905),
                                          (2, 131072, 990, 1000), (400, 20000, 1e4, 1e4 + 40)])
def test_logprobs_of_rising_rows_far_from_zero(rows, V, lo, hi, dtype):
    """Rows that rise past 1024, where exponents are formed in another way, past it, or
    stay below: up to 8 references a thread, each changed by a factor that is off by
    2^-19.2 (its exponent, below 2^5, rounded, and its exponential), and three joins off by as much
    and five sums; 2^-18 for the thread's own sums as above: together below 2^-15.5."""
    i = torch.arange(V, device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = (lo + (hi - lo) * i / V + 0.5 * torch.randn((rows, V), generator=g, device="cuda", dtype=torch.float64)).to(dtype)
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    got = run_logprobs(x, tok, 5)
    lp, rank, ent, ids, tlp = R.logprob_reference(x, tok, 5)
    off = 2.0 ** -15.5
    for a, b, t in ((got[0], lp, off), (got[4], tlp, off), (got[2], ent, off * (math.log(V) + 3))):
        assert ((a.double() - b).abs() <= t + 2.0 ** -22 * b.abs()).all()
    assert torch.equal(got[1].long(), rank.long()) and torch.equal(got[3].long(), ids)


@pytest.mark.parametrize("graph", [False, True])
def test_ragged_step_ranks(graph):
    """The four calls one after another, eager and captured, with the ranks among the
    outputs of the last: counts of what lies above the token in the step's own logits."""
    pa = _pa()
    rng = np.random.default_rng(64)
    B, T, NQ, NKV, V, NB = 3, 40, 8, 2, 777, 6
    f = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    act, new_act, lens, head, new_head = z(B), z(B), z(B), z(1), z(1)
    bt, pool = torch.full((B, 2), -1, dtype=torch.int32, device="cuda"), torch.arange(NB, dtype=torch.int32, device="cuda")
    slots, pos, tb, cu, tok = z(T), z(T), z(T), z(B + 1), z(T)
    kc, vc, ks = z(NB, BS, NKV, D, dt=torch.uint8), z(NB, BS, NKV, D, dt=torch.uint8), z(NB, BS, NKV, dt=torch.float32)
    qc, qs, vs = z(T, NQ, D, dt=torch.uint8), z(T, NQ, dt=torch.float32), torch.full((B, NKV, D), 0.02, device="cuda")
    ang, w, w_out = f(300, 16), 1 + f(D) / 8, f(NQ * D, V) / 30
    cs, qkv = torch.cat([ang.cos(), ang.sin()], 1), z(T, NQ + 2 * NKV, D, dt=torch.float32)
    out, logits = z(T, NQ, D, dt=torch.bfloat16), z(T, V, dt=torch.float32)
    lp, rank, ent, ids, tlp = z(T, dt=torch.float32), z(T), z(T, dt=torch.float32), z(T, 4), z(T, 4, dt=torch.float32)
    ws = pa.WindowWorkspace(T, NQ, NKV)

    def step():
        pa.plan_batch(act, lens, pool, head, bt, slots, pos, tb, cu, new_act, new_head, num_blocks=NB)
        pa.qkv_norm_mrope_append(qkv[:, :NQ], qkv[:, NQ:NQ + NKV], qkv[:, NQ + NKV:], w, w, cs, pos[None], qc, qs, kc, vc,
                                 slots, ks, vs, tb, pair_axis=[0] * 16, layout=pa.LAYOUT_BSND)
        pa.window_attention(qc, qs, kc, ks, vc, vs, bt, new_act, cu, out, window=20, sinks=2, layout=pa.LAYOUT_BSND,
                            workspace=ws)
        torch.matmul(out.float().view(T, -1), w_out, out=logits)
        pa.token_logprobs(logits, tok, lp, ranks=rank, entropy=ent, top_ids=ids, top_logprobs=tlp)

    call = step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                         # (of no tokens)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        call = g.replay
    for new in ([30, 1, 0], [1, 5, 33]):
        lens.copy_(_i32(*new))
        qkv.copy_(f(T, NQ + 2 * NKV, D))
        tok.copy_(torch.from_numpy(rng.integers(0, V, T).astype(np.int32)))
        rank.fill_(-7)
        call()
        torch.cuda.synchronize()
        n = sum(new)
        assert ws.error_flags() == 0 and int(cu[-1]) == n
        own = logits.gather(1, tok.long()[:, None])
        assert torch.equal(rank[:n].long(), (logits > own).sum(-1)[:n]) and rank[:n].float().std() > 100
        check_logprobs(logits[:n], tok[:n], 4, tuple(t[:n] for t in (lp, rank, ent, ids, tlp)))
        act.copy_(new_act)
        head.copy_(new_head)
