"""Host-side checks of the speculative decode step's entry points (no GPU
needed): every refusal comes before anything is enqueued."""
import ctypes

import pytest

from tests.test_abi import _buf

P = ctypes.c_void_p
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import fp8_paged_kv_block_gb300 as pa
    pa.build()
    return pa.lib()


def caller(fn, order, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a)
        a.update(kw)
        return fn(*[a[k] for k in order])
    return call


def test_append_refusals(L):
    fake = _buf()
    names = ("q k v dt qs ks vs qw kw wdt eps cs rd maxpos inter pos pdt qc qsc kc vc slots sdt ksc vsc tb nb T NQ "
             "NKV D NB BS layout stream").split()
    d = {n: fake for n in "q k v qw kw cs pos qc qsc kc vc slots ksc vsc tb".split()}
    d.update(dt=1, qs=2048, ks=2048, vs=2048, wdt=1, eps=1e-5, rd=64, maxpos=100, inter=0, pdt=0, sdt=0, nb=2, T=4,
             NQ=8, NKV=2, D=128, NB=4, BS=128, layout=0, stream=None)
    call = caller(L.pa_fp8_qkv_norm_rope_append, names, d)
    for n in "q k v qc qsc kc vc slots ksc vsc tb cs pos".split():
        assert call(**{n: None}) == 1, n
    assert call(T=0) == 0                                  # nothing to do
    assert call(T=0, cs=None, pos=None, rd=0, qw=None, kw=None) == 0
    assert call(T=0, **{n: None for n in "q k v qc qsc slots tb pos".split()}) == 0
    assert call(T=0, kc=None) == 1 and call(T=0, cs=None) == 1 and call(T=0, layout=2) == 2
    for bad in (dict(T=-1), dict(NQ=0), dict(NKV=0), dict(D=0), dict(NB=0), dict(BS=0), dict(nb=0), dict(dt=2),
                dict(wdt=-1), dict(sdt=2), dict(pdt=2), dict(layout=2), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
                dict(maxpos=0), dict(rd=-16), dict(rd=144), dict(qs=2044), dict(dt=0, vs=2046),
                dict(q=P(fake.value + 2)), dict(kc=P(fake.value + 4)), dict(qw=P(fake.value + 8))):
        assert call(**bad) == 2, bad
    for bad in (dict(D=96), dict(D=512), dict(rd=8), dict(rd=4, inter=1), dict(T=1 << 40)):
        assert call(**bad) == 5, bad
    assert b"head rows" in L.pa_last_error()


def test_tree_decode_refusals(L):
    fake = _buf()
    n = ctypes.c_size_t(0)
    size = L.pa_fp8_tree_decode_workspace_size
    assert size(4, 8, 96, 8, 128, None) == 1
    assert size(4, 8, 96, 8, 128, ctypes.byref(n)) == 0 and n.value >= 256 and n.value % 256 == 0
    for bad, st in (((-1, 8, 96, 8, 128), 2), ((4, 0, 96, 8, 128), 2), ((4, 8, 96, 7, 128), 2), ((4, 8, 0, 8, 128), 2),
                    ((4, 8, 96, 8, 64), 5), ((1025, 8, 96, 8, 128), 5), ((4, 129, 96, 8, 128), 5),
                    ((4, 8, 129, 1, 128), 5)):
        assert size(*bad, ctypes.byref(n)) == st, bad
    size(4, 8, 96, 8, 128, ctypes.byref(n))
    names = "q qs kc ks vc vs bt act len mask ms out B S1 NQ NKV D BS NB MB layout scale ws wsb stream".split()
    d = {k: fake for k in "q qs kc ks vc vs bt act len mask out".split()}
    d.update(ms=64, B=4, S1=8, NQ=96, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, scale=0.08,
             ws=P((fake.value + 255) & ~255), wsb=n.value, stream=None)
    call = caller(L.pa_fp8_tree_decode, names, d)
    for k in "q qs kc ks vc vs bt act mask out".split():
        assert call(**{k: None}) == 1, k
    assert call(B=0) == 0 and call(B=0, **{k: None for k in "q qs vs bt act len mask out ws".split()}) == 0
    assert call(B=0, kc=None) == 1 and call(B=0, layout=3) == 2
    for bad in (dict(B=-1), dict(NB=0), dict(MB=0), dict(layout=3), dict(scale=NAN), dict(scale=INF), dict(ms=-1),
                dict(NQ=97), dict(q=P(fake.value + 8)), dict(out=P(fake.value + 2)),
                dict(ws=P(((fake.value + 255) & ~255) + 16))):
        assert call(**bad) == 2, bad
    for bad in (dict(BS=64), dict(D=64), dict(S1=129), dict(B=1025), dict(MB=1 << 30), dict(NB=1 << 40)):
        assert call(**bad) == 5, bad
    assert call(ws=None) == 3
    assert call(wsb=n.value - 1) == 3 and b"needed" in L.pa_last_error()


def test_verify_refusals(L):
    fake = _buf()
    names = "p q tok par u len B S1 V acc path new stream".split()
    d = {k: fake for k in "p q tok par u len acc path new".split()}
    d.update(B=2, S1=4, V=1000, stream=None)
    call = caller(L.pa_tree_verify, names, d)
    for k in "p tok par u acc path new".split():
        assert call(**{k: None}) == 1, k
    assert call(B=0) == 0 and call(B=0, **{k: None for k in "p q tok par u len acc path new".split()}) == 0
    for bad in (dict(B=-1), dict(S1=0), dict(V=0), dict(p=P(fake.value + 2)), dict(new=P(fake.value + 1))):
        assert call(**bad) == 2, bad
    for bad in (dict(S1=1025), dict(V=262145), dict(B=(1 << 24) + 1)):
        assert call(**bad) == 5, bad


def test_keep_path_refusals(L):
    fake, other = _buf(), _buf()
    names = "kc vc ks bt act len path acc new B S1 NKV D BS NB MB layout stream".split()
    d = {k: fake for k in "kc vc ks bt act len path acc".split()}
    d.update(new=other, B=2, S1=4, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, stream=None)
    call = caller(L.pa_fp8_cache_keep_path, names, d)
    for k in "kc vc ks bt act path acc new".split():
        assert call(**{k: None}) == 1, k
    assert call(B=0) == 0 and call(B=0, **{k: None for k in "bt act len path acc new".split()}) == 0
    assert call(B=0, kc=None) == 1
    for bad in (dict(B=-1), dict(S1=0), dict(NKV=0), dict(D=0), dict(BS=0), dict(NB=0), dict(MB=0), dict(layout=9),
                dict(new=fake), dict(kc=P(fake.value + 8))):
        assert call(**bad) == 2, bad
    for bad in (dict(D=24), dict(D=8208), dict(S1=1025)):
        assert call(**bad) == 5, bad


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """The binding's checks come before the library is asked."""
    torch = pytest.importorskip("torch")
    import fp8_paged_kv_block_gb300 as pa
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.tree_verify(z(1, 2, 8), None, z(1, 2, **i32), z(1, 2, **i32), z(1, 2), z(1, **i32), z(1, 2, **i32),
                       z(1, 2, **i32))
    with pytest.raises(ValueError, match="CUDA"):
        pa.cache_keep_path(z(1, 128, 1, 128, dtype=torch.uint8), z(1, 128, 1, 128, dtype=torch.uint8),
                           z(1, 128, 1), z(1, 1, **i32), z(1, **i32), z(1, 2, **i32), z(1, **i32), z(1, **i32))
    with pytest.raises(TypeError):
        pa.tree_decode(None, *[z(1)] * 9, S1=1)
    with pytest.raises(ValueError, match="CUDA"):
        pa.qkv_norm_rope_append(*[z(1, 1, 128)] * 3, None, None, None, None, *[z(1)] * 8)


class _Stream:
    """What the binding takes from a torch stream, without a GPU."""
    cuda_stream = 0


def _on_host(monkeypatch):
    """The binding with host tensors let through and nothing launched: what it
    refuses beyond the tensors' place can then be tested without a GPU."""
    import fp8_paged_kv_block_gb300 as pa
    monkeypatch.setattr(pa, "_need", lambda t, name, dtype=None, contiguous=True: _need_dtype(t, name, dtype))
    monkeypatch.setattr(pa, "_one_device", lambda **kw: None)
    return pa


def _need_dtype(t, name, dtype):
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s has dtype %s" % (name, t.dtype))


def test_keep_path_wants_a_layout(L, monkeypatch):
    """A cache [NB, 128, 8, 128] reads as 8 heads or as 128: no default decides."""
    torch = pytest.importorskip("torch")
    pa = _on_host(monkeypatch)
    i32 = dict(dtype=torch.int32)
    cache = [torch.zeros((3, 128, 8, 128), dtype=torch.uint8) for _ in range(2)] + [torch.zeros((3, 128, 8))]
    args = cache + [torch.zeros((2, 2), **i32), torch.zeros(2, **i32), torch.zeros((2, 4), **i32),
                    torch.zeros(2, **i32), torch.zeros(2, **i32)]
    for call in (pa.cache_keep_path, pa.prepare_cache_keep_path):
        with pytest.raises(TypeError, match="layout"):
            call(*args, stream=_Stream())
    for layout in (pa.LAYOUT_BSND, pa.LAYOUT_BNBD):
        pa.prepare_cache_keep_path(*args, layout=layout, stream=_Stream())


def test_outputs_that_overlap_inputs_are_refused(L):
    """The kernels read their inputs while outputs are already written."""
    pool = _buf().value
    at = lambda i: P(pool + 4096 * i)  # noqa: E731
    names = "p q tok par u len B S1 V acc path new stream".split()
    d = {k: at(i) for i, k in enumerate("p q tok par u len acc path new".split())}
    d.update(S1=4, V=100, B=2, stream=None)               # 8 rows: 3200 bytes of probabilities
    verify = caller(L.pa_tree_verify, names, d)
    for out, size in (("acc", 8), ("path", 32), ("new", 32)):
        for i, other in enumerate("p q tok par u len acc path new".split()):
            if other == out:
                continue
            for off in (0, 4, -size + 4):
                assert verify(**{out: P(d[other].value + off)}) == 2, (out, other, off)
                assert b"overlap" in L.pa_last_error()
    names = "kc vc ks bt act len path acc new B S1 NKV D BS NB MB layout stream".split()
    d = {k: at(i) for i, k in enumerate("kc vc ks bt act len path acc new".split())}
    d.update(B=2, S1=4, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, stream=None)
    keep = caller(L.pa_fp8_cache_keep_path, names, d)
    for other in "bt act len path acc".split():
        for off in (0, 4, -4):
            assert keep(new=P(d[other].value + off)) == 2, (other, off)
            assert b"overlap" in L.pa_last_error()


def test_append_of_tokens_past_32_bits_is_refused(L):
    """Offsets within a token are 32 bits."""
    fake = _buf()
    names = ("q k v dt qs ks vs qw kw wdt eps cs rd maxpos inter pos pdt qc qsc kc vc slots sdt ksc vsc tb nb T NQ "
             "NKV D NB BS layout stream").split()
    d = {n: fake for n in "q k v qw kw cs pos qc qsc kc vc slots ksc vsc tb".split()}
    d.update(dt=1, qs=2048, ks=2048, vs=2048, wdt=1, eps=1e-5, rd=64, maxpos=100, inter=0, pdt=0, sdt=0, nb=2, T=1,
             NQ=8, NKV=2, D=128, NB=4, BS=128, layout=0, stream=None)
    call = caller(L.pa_fp8_qkv_norm_rope_append, names, d)
    for bad in (dict(NQ=1 << 24), dict(NKV=1 << 24), dict(NQ=1 << 23, D=256), dict(NKV=1 << 25, D=64)):
        assert call(**bad) == 5 and b"2^31" in L.pa_last_error(), bad
    assert call(T=0, NQ=(1 << 24) - 1) == 0


def test_elements_off_their_alignment_are_refused(L):
    """A misaligned address is a fault on the GPU."""
    fake, other = _buf(), _buf()
    names = ("q k v dt qs ks vs qw kw wdt eps cs rd maxpos inter pos pdt qc qsc kc vc slots sdt ksc vsc tb nb T NQ "
             "NKV D NB BS layout stream").split()
    d = {n: fake for n in "q k v qw kw cs pos qc qsc kc vc slots ksc vsc tb".split()}
    d.update(dt=1, qs=2048, ks=2048, vs=2048, wdt=1, eps=1e-5, rd=64, maxpos=100, inter=0, pdt=0, sdt=0, nb=2, T=0,
             NQ=8, NKV=2, D=128, NB=4, BS=128, layout=0, stream=None)
    call = caller(L.pa_fp8_qkv_norm_rope_append, names, d)
    for n in "pos slots tb qsc ksc".split():
        assert call(**{n: P(fake.value + 2)}) == 2, n
    assert call(pos=P(fake.value + 4), slots=P(fake.value + 4)) == 0
    assert call(pos=P(fake.value + 4), pdt=1) == 2 and call(slots=P(fake.value + 4), sdt=1) == 2
    names = "q qs kc ks vc vs bt act len mask ms out B S1 NQ NKV D BS NB MB layout scale ws wsb stream".split()
    d = {k: fake for k in "q qs kc ks vc vs bt act len mask out".split()}
    d.update(ms=64, B=0, S1=8, NQ=96, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, scale=0.08, ws=None, wsb=0,
             stream=None)
    call = caller(L.pa_fp8_tree_decode, names, d)
    assert call(mask=P(fake.value + 1)) == 0
    for n in "qs ks bt act len".split():
        assert call(**{n: P(fake.value + 2)}) == 2 and b"4-byte" in L.pa_last_error(), n
    names = "kc vc ks bt act len path acc new B S1 NKV D BS NB MB layout stream".split()
    d = {k: fake for k in "kc vc ks bt act len path acc".split()}
    d.update(new=other, B=0, S1=4, NKV=8, D=128, BS=128, NB=16, MB=4, layout=0, stream=None)
    call = caller(L.pa_fp8_cache_keep_path, names, d)
    assert call() == 0
    for n in "ks bt act len path acc new".split():
        assert call(**{n: P(d[n].value + 2)}) == 2 and b"misaligned" in L.pa_last_error(), n


def test_append_writes_e4m3_codes_into_nothing_else(L, monkeypatch):
    torch = pytest.importorskip("torch")
    pa = _on_host(monkeypatch)
    T, NQ, NKV, D = 3, 4, 2, 128

    def prepare(**dt):
        z = lambda n, *s: torch.zeros(s, dtype=dt.get(n, torch.uint8))  # noqa: E731
        f = torch.zeros
        return pa.prepare_qkv_norm_rope_append(
            f(T, NQ, D), f(T, NKV, D), f(T, NKV, D), None, None, None, None, z("q_codes", T, NQ, D), f(T, NQ),
            z("key_cache", 2, 128, NKV, D), z("value_cache", 2, 128, NKV, D), f(T, dtype=torch.int32),
            f(2, 128, NKV), f(1, NKV, D), f(T, dtype=torch.int32), layout=pa.LAYOUT_BSND, stream=_Stream())
    for n in ("q_codes", "key_cache", "value_cache"):
        prepare(**{n: torch.float8_e4m3fn})
        with pytest.raises(TypeError, match=n):
            prepare(**{n: torch.float8_e5m2})


def test_prepared_calls_refuse_another_current_device(L, monkeypatch):
    """On a default stream the launch goes to the current device."""
    torch = pytest.importorskip("torch")
    pa = _on_host(monkeypatch)
    ran = []
    current = [0]
    i32 = dict(dtype=torch.int32)
    call = pa.prepare_cache_keep_path(
        torch.zeros((1, 128, 1, 128), dtype=torch.uint8), torch.zeros((1, 128, 1, 128), dtype=torch.uint8),
        torch.zeros((1, 128, 1)), torch.zeros((1, 1), **i32), torch.zeros(1, **i32), torch.zeros((1, 2), **i32),
        torch.zeros(1, **i32), torch.zeros(1, **i32), layout=pa.LAYOUT_BSND, stream=_Stream())
    call._call = lambda stream: ran.append(stream.value) or 0
    call._device, call._current, call._several = 0, lambda: current[0], True
    call()
    current[0] = 1
    with pytest.raises(ValueError, match="current device is cuda:1"):
        call()
    other = _Stream()
    other.cuda_stream = 4096
    call(other)                                          # (the runtime itself tells such a launch's device)
    assert ran == [None, 4096]
