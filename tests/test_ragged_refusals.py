"""Host-side checks of the ragged serving step's entry points (no GPU needed): every
refusal comes before anything is enqueued."""
import ctypes

import pytest

from tests.test_abi import _buf
from tests.test_draft_refusals import L, P, _on_host, _Stream, caller  # noqa: F401

NAN, INF = float("nan"), float("inf")


def test_plan_refusals(L):  # noqa: F811
    pool = _buf().value
    at = lambda i: P(pool + 512 * i)  # noqa: E731
    names = "act lens pool head bt slots sdt pos tb cu nact nhead B T P NB BS W stream".split()
    tensors = "act lens pool head bt slots pos tb cu nact nhead".split()
    d = {k: at(i) for i, k in enumerate(tensors)}
    d.update(sdt=0, B=4, T=8, P=16, NB=16, BS=128, W=4, stream=None)
    call = caller(L.pa_plan_batch, names, d)
    for n in tensors:
        assert call(**{n: None}) == 1, n
    for bad in (dict(B=-1), dict(T=-1), dict(P=-1), dict(NB=0), dict(BS=0), dict(W=0), dict(sdt=2),
                dict(pos=P(pool + 2)), dict(slots=P(pool + 4096 + 4), sdt=1)):
        assert call(**bad) == 2, bad
    for bad in (dict(B=1025), dict(T=1 << 31), dict(P=1 << 31), dict(W=1 << 30), dict(NB=1 << 24)):
        assert call(**bad) == 5, bad
    # outputs over inputs and over one another, by one element too
    sizes = dict(act=16, lens=16, pool=64, head=4, bt=64, slots=32, pos=32, tb=32, cu=20, nact=16, nhead=4)
    for out in "bt slots pos tb cu nact nhead".split():
        for other in tensors:
            if other == out:
                continue
            for off in (0, sizes[other] - 4, 4 - sizes[out]):
                assert call(**{out: P(d[other].value + off)}) == 2, (out, other, off)
                assert b"overlap" in L.pa_last_error()


def test_mrope_append_refusals(L):  # noqa: F811
    fake = _buf()
    names = ("q k v dt qs ks vs qw kw wdt eps cs rd maxpos inter pos pdt A astep axis qc qsc kc vc slots sdt ksc vsc tb "
             "nb T NQ NKV D NB BS layout stream").split()
    axis = (ctypes.c_uint8 * 32)(*([0] * 8 + [1] * 12 + [2] * 12))
    d = {n: fake for n in "q k v qw kw cs pos qc qsc kc vc slots ksc vsc tb".split()}
    d.update(dt=1, qs=2048, ks=2048, vs=2048, wdt=1, eps=1e-5, rd=64, maxpos=100, inter=0, pdt=0, A=3, astep=4,
             axis=ctypes.addressof(axis), sdt=0, nb=2, T=4, NQ=8, NKV=2, D=128, NB=4, BS=128, layout=0, stream=None)
    call = caller(L.pa_fp8_qkv_norm_mrope_append, names, d)
    for n in "q k v qc qsc kc vc slots ksc vsc tb cs pos axis".split():
        assert call(**{n: None}) == 1, n
    assert call(T=0) == 0 and call(T=0, rd=0, axis=None, cs=None, pos=None) == 0
    for bad in (dict(A=0), dict(A=-1), dict(A=2), dict(astep=3), dict(astep=-1), dict(T=-1), dict(rd=-16), dict(rd=144),
                dict(maxpos=0), dict(layout=2), dict(eps=NAN), dict(qs=2044), dict(pos=P(fake.value + 2))):
        assert call(**bad) == 2, bad
    assert call(A=2, T=0) == 2 and b"pair 20 on axis 2 of 2" in L.pa_last_error()
    for bad in (dict(A=5), dict(D=96), dict(rd=8)):
        assert call(**bad) == 5, bad


def test_window_attention_refusals(L):  # noqa: F811
    fake = _buf()
    n = ctypes.c_size_t(0)
    size = L.pa_fp8_window_attention_workspace_size
    assert size(8, 96, 8, 128, None) == 1
    assert size(8, 96, 8, 128, ctypes.byref(n)) == 0 and n.value >= 256 and n.value % 256 == 0
    small = n.value
    assert size(1 << 30, 96, 8, 128, ctypes.byref(n)) == 0 and n.value >= small
    for bad, st in (((0, 96, 8, 128), 2), ((-1, 96, 8, 128), 2), ((8, 96, 7, 128), 2), ((8, 0, 8, 128), 2),
                    ((8, 96, 8, 64), 5), ((8, 129, 1, 128), 5)):
        assert size(*bad, ctypes.byref(n)) == st, bad
    names = "q qs kc ks vc vs bt act cu out B T most NQ NKV D BS NB MB layout win sinks scale ws wsb stream".split()
    d = {k: fake for k in "q qs kc ks vc vs bt act cu out".split()}
    ws = (fake.value + 255) & ~255
    d.update(B=4, T=20, most=8, NQ=96, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, win=100, sinks=4, scale=0.08,
             ws=P(ws), wsb=small, stream=None)
    call = caller(L.pa_fp8_window_attention, names, d)
    for k in "q qs kc ks vc vs bt act cu out".split():
        assert call(**{k: None}) == 1, k
    rest = {k: None for k in "q qs vs bt act cu out ws".split()}
    assert call(B=0) == 0 and call(T=0) == 0 and call(B=0, **rest) == 0 and call(T=0, **rest) == 0
    assert call(B=0, kc=None) == 1 and call(T=0, layout=3) == 2
    for bad in (dict(B=-1), dict(T=-1), dict(most=0), dict(NB=0), dict(MB=0), dict(layout=3), dict(scale=NAN),
                dict(scale=INF), dict(win=-1), dict(sinks=-1), dict(NQ=97), dict(q=P(fake.value + 8)),
                dict(out=P(fake.value + 2)), dict(ws=P(ws + 16))):
        assert call(**bad) == 2, bad
    for k in "qs ks bt act cu".split():
        assert call(**{k: P(fake.value + 2)}) == 2 and b"4-byte" in L.pa_last_error(), k
    for bad in (dict(BS=64), dict(D=64), dict(B=1025), dict(MB=1 << 30), dict(NB=1 << 40), dict(T=1 << 31),
                dict(T=(1 << 31) // 96, MB=(1 << 17) - 1)):
        assert call(**bad) == 5, bad
    assert call(ws=None) == 3
    assert call(wsb=small - 1) == 3 and b"needed" in L.pa_last_error()
    apart = {k: P((i + 1) << 36) for i, k in enumerate("q qs kc ks vc vs bt act cu out".split())}
    for k, size in dict(q=20 * 96 * 128, qs=20 * 96 * 4, kc=16 * 8 * 128 ** 2, ks=16 * 8 * 128 * 4, vc=16 * 8 * 128 ** 2,
                        vs=4 * 8 * 128 * 4, bt=64, act=16, cu=20).items():
        for at in (apart[k].value + size - 4 & ~15, apart[k].value - 20 * 96 * 256 + 16):
            assert call(**{**apart, "out": P(at)}) == 2 and b"overlaps" in L.pa_last_error(), k


def test_token_logprobs_refusals(L):  # noqa: F811
    fake = _buf()
    names = "x dt step tok tdt R V lp rank ent k ids tlp stream".split()
    d = {k: fake for k in "x tok lp rank ent ids tlp".split()}
    d.update(dt=1, step=1000, tdt=0, R=4, V=1000, k=5, stream=None)
    call = caller(L.pa_token_logprobs, names, d)
    for k in "x tok lp ids tlp".split():
        assert call(**{k: None}) == 1, k
    assert call(R=0) == 0 and call(R=0, **{k: None for k in "x tok lp rank ent ids tlp".split()}) == 0
    for bad in (dict(R=-1), dict(V=0), dict(k=-1), dict(k=6, V=5), dict(dt=2), dict(tdt=2), dict(step=999),
                dict(x=P(fake.value + 1)), dict(x=P(fake.value + 2), dt=0), dict(lp=P(fake.value + 2)),
                dict(tok=P(fake.value + 4), tdt=1)):
        assert call(**bad) == 2, bad
    for bad in (dict(k=33), dict(V=(1 << 31) - 1, step=1 << 40), dict(R=1 << 40)):
        assert call(**bad) == 5, bad
    apart = {k: P((i + 1) << 36) for i, k in enumerate("x tok lp rank ent ids tlp".split())}
    for k, size in dict(x=4 * (3 * 1000 + 1000) // 2, tok=16, lp=16, rank=16, ent=16, ids=80, tlp=80).items():
        for o, n in dict(lp=16, rank=16, ent=16, ids=80, tlp=80).items():
            if o != k:
                for at in (apart[k].value + size - 4, apart[k].value - n + 4):
                    assert call(**{**apart, o: P(at)}) == 2 and b"overlap" in L.pa_last_error(), (k, o)


def test_binding_refuses_wrong_shapes_and_host_tensors(L, monkeypatch):  # noqa: F811
    torch = pytest.importorskip("torch")
    import fp8_paged_kv_block_gb300 as pa
    i32 = dict(dtype=torch.int32)
    z = lambda *s, **k: torch.zeros(s, **k)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pa.token_logprobs(z(2, 9), z(2, **i32), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        pa.plan_batch(*[z(2, **i32)] * 11, num_blocks=4)
    with pytest.raises(ValueError, match="CUDA"):
        pa.window_attention(*[z(1, 1, 128, dtype=torch.uint8)] * 10, window=4)
    pa = _on_host(monkeypatch)
    s = _Stream()

    def plan(**kw):
        a = dict(kv_act_seqs=z(2, **i32), new_lens=z(2, **i32), pool=z(5, **i32), pool_head=z(1, **i32),
                 block_table=z(2, 4, **i32), slot_mapping=z(7, **i32), positions=z(7, **i32), token_batch=z(7, **i32),
                 cu_tokens=z(3, **i32), new_act_seqs=z(2, **i32), new_pool_head=z(1, **i32))
        a.update(kw)
        return pa.prepare_plan_batch(**a, num_blocks=9, stream=s)
    plan()
    plan(slot_mapping=z(7, dtype=torch.int64))
    for bad in (dict(new_lens=z(3, **i32)), dict(cu_tokens=z(2, **i32)), dict(positions=z(6, **i32)),
                dict(block_table=z(2, **i32)), dict(pool_head=z(2, **i32)), dict(pool=z(1, 5, **i32))):
        with pytest.raises(ValueError):
            plan(**bad)
    for bad in (dict(slot_mapping=z(7)), dict(pool=z(5, dtype=torch.int64))):
        with pytest.raises(TypeError):
            plan(**bad)

    def logp(x=None, tok=None, **kw):
        return pa.prepare_token_logprobs(z(3, 9) if x is None else x, z(3, **i32) if tok is None else tok, z(3), stream=s,
                                         **kw)
    logp()
    logp(z(3, 16)[:, :9], ranks=z(3, **i32), entropy=z(3), top_ids=z(3, 2, **i32), top_logprobs=z(3, 2))
    for bad in (dict(x=z(9)), dict(x=z(9, 3).T), dict(x=z(1, 9).expand(3, 9)), dict(tok=z(4, **i32)),
                dict(top_ids=z(3, 2, **i32)), dict(top_ids=z(3, 2, **i32), top_logprobs=z(3, 1)), dict(ranks=z(2, **i32))):
        with pytest.raises(ValueError):
            logp(**bad)
    for bad in (dict(x=z(3, 9, dtype=torch.float16)), dict(tok=z(3)), dict(entropy=z(3, **i32))):
        with pytest.raises(TypeError):
            logp(**bad)

    u8 = dict(dtype=torch.uint8)

    def window(**kw):
        a = dict(q=z(6, 4, 128, **u8), q_scale=z(6, 4), k_cache=z(3, 128, 2, 128, **u8), k_scale=z(3, 128, 2),
                 v_cache=z(3, 128, 2, 128, **u8), v_scale=z(2, 2, 128), block_table=z(2, 4, **i32),
                 kv_act_seqs=z(2, **i32), cu_tokens=z(3, **i32), out=z(6, 4, 128, dtype=torch.bfloat16), window=5, sinks=0,
                 workspace=type("W", (), dict(buf=z(512), nbytes=512))())
        a.update(kw)
        return pa.prepare_window_attention(**a, stream=s)
    window()
    window(window=None)
    for bad in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(cu_tokens=z(2, **i32)), dict(out=z(
            5, 4, 128, dtype=torch.bfloat16)), dict(q_scale=z(6, 3)), dict(k_scale=z(3, 128)), dict(v_scale=z(1, 2, 128)),
                dict(block_table=z(3, 4, **i32)), dict(q=z(6, 512, **u8)), dict(layout=pa.LAYOUT_BNBD)):
        with pytest.raises(ValueError):
            window(**bad)
    with pytest.raises(TypeError):
        window(k_cache=z(3, 128, 2, 128, dtype=torch.float8_e5m2))

    def mrope(positions=None, pair_axis=(0, 1) * 16, cos_sin=None):
        return pa.prepare_qkv_norm_mrope_append(
            z(3, 4, 128), z(3, 2, 128), z(3, 2, 128), None, None, z(9, 64) if cos_sin is None else cos_sin,
            z(2, 3, **i32) if positions is None else positions, z(3, 4, 128, **u8), z(3, 4), z(2, 128, 2, 128, **u8),
            z(2, 128, 2, 128, **u8), z(3, **i32), z(2, 128, 2), z(1, 2, 128), z(3, **i32), pair_axis=pair_axis,
            layout=pa.LAYOUT_BSND, stream=s)
    mrope()
    mrope(z(2, 8, **i32)[:, :3])
    for bad in (dict(positions=z(3, **i32)), dict(positions=z(2, 4, **i32)), dict(positions=z(3, 2, **i32).T),
                dict(positions=z(1, 3, **i32).expand(2, 3)), dict(positions=z(1, 3, **i32)), dict(pair_axis=[0] * 31),
                dict(pair_axis=[0] * 31 + [-1])):
        with pytest.raises(ValueError):
            mrope(**bad)
    with pytest.raises(TypeError):
        mrope(pair_axis=None)


def test_empty_ranges_overlap_nothing(L):  # noqa: F811
    """What has no elements may lie anywhere, an empty slice of another tensor among
    it. (Each call has one overlap that counts, tested behind the empty ranges, so
    that it is refused for that one and launches nothing.)"""
    pool = _buf().value
    at = lambda i: P(pool + 512 * i)  # noqa: E731
    names = "act lens pool head bt slots sdt pos tb cu nact nhead B T P NB BS W stream".split()
    d = {k: at(i) for i, k in enumerate("act lens pool head bt slots pos tb cu nact nhead".split())}
    d.update(sdt=0, B=4, T=8, P=0, NB=16, BS=128, W=4, stream=None, tb=d["cu"])
    call = caller(L.pa_plan_batch, names, d)
    for off in (0, 16):                                  # a used-up pool, at the table's begin and inside it
        assert call(pool=P(d["bt"].value + off)) == 2 and b"outputs overlap" in L.pa_last_error(), off
    # no tokens: their tensors anywhere
    none = {k: P(d["bt"].value + 16) for k in "slots pos tb".split()}
    assert call(T=0, nhead=d["head"], **none) == 2 and b"an output overlaps an input" in L.pa_last_error()
    names = "x dt step tok tdt R V lp rank ent k ids tlp stream".split()
    d = {k: P((i + 1) << 36) for i, k in enumerate("x tok lp rank ent ids tlp".split())}
    d.update(dt=1, step=1000, tdt=0, R=4, V=1000, k=0, stream=None, rank=d["tok"])
    call = caller(L.pa_token_logprobs, names, d)
    for off in (0, 8, 1):                                # (not used with 0 alternatives: any address)
        stale = P(d["lp"].value + off)
        assert call(ids=stale, tlp=stale) == 2 and b"an output overlaps an input" in L.pa_last_error(), off
