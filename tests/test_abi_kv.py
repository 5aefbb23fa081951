"""CPU checks of the cache entry points: every refusal happens on the host.

The addresses are never dereferenced (see test_abi.py)."""
import copy
import ctypes

import pytest

import quantized_gemm_nvfp4_amd as q

OK, INVALID, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = ctypes.c_void_p
BASE = [P(0x10000000 * (i + 1)) for i in range(12)]
KC, KS, VC, VS, KGP, VGP, X, Y, Z, W, SL, T = BASE


def err():
    return q.lib().nvfp4_last_error().decode()


def cache(pages=4, ps=16, heads=2, d=128, **kw):
    f = dict(k_codes=KC, k_scales=KS, v_codes=VC, v_scales=VS, k_gscale=KGP, v_gscale=VGP, num_pages=pages,
             page_size=ps, kv_heads=heads, head_dim=d)
    f.update(kw)
    c = q._CacheStruct(*[v.value if isinstance(v, P) else v for v in f.values()])
    return ctypes.byref(c)


def write(c=None, k=X, ks=256, v=Y, vs=256, slots=SL, tokens=0):
    return q.lib().nvfp4_kv_write(c or cache(), k, ks, v, vs, slots, tokens, None)


def read(c=None, slots=SL, tokens=0, k=X, v=Y):
    return q.lib().nvfp4_kv_read(c or cache(), slots, tokens, k, v, None)


def test_cache_description():
    assert write(tokens=0) == OK and read(tokens=0) == OK
    assert q.lib().nvfp4_kv_write(None, X, 256, Y, 256, SL, 1, None) == INVALID and "cache" in err()
    for ps in (0, 8, 24, 8192, -16):
        assert write(cache(ps=ps)) in (SHAPE, INVALID) and "page_size" in err()
    for d in (16, 96, 512):
        assert write(cache(d=d)) == UNSUP and "head_dim" in err()
    assert write(cache(heads=0)) == UNSUP
    assert write(cache(pages=-1)) == INVALID
    assert write(cache(pages=1 << 31)) == UNSUP
    assert write(cache(pages=1 << 30, heads=64, ps=4096)) == UNSUP
    assert write(cache(v_codes=None)) == INVALID and "v_codes" in err()
    assert write(cache(k_scales=P(0x10008))) == ALIGN and "k_scales" in err()
    assert write(cache(k_gscale=None)) == INVALID and "k_gscale" in err()
    assert write(cache(v_gscale=P(0x10002))) == ALIGN


def test_write_and_read_refusals():
    assert write(k=None, tokens=3) == INVALID and "k is" in err()
    assert write(v=P(0x70000008), tokens=3) == ALIGN
    assert write(ks=248, tokens=3) == SHAPE and "stride" in err()
    assert write(vs=260, tokens=3) == ALIGN
    assert write(slots=None, tokens=3) == INVALID
    assert write(slots=P(0x10004), tokens=3) == ALIGN
    assert write(tokens=-1) == INVALID
    assert write(tokens=1 << 30) == UNSUP
    assert write(k=KC, tokens=3) == INVALID and "overlap" in err()
    assert write(slots=VS, tokens=3) == INVALID and "overlap" in err()
    assert read(k=Y, tokens=3) == INVALID and "overlap" in err()
    assert read(v=KC, tokens=3) == INVALID and "overlap" in err()
    assert read(v=KGP, tokens=3) == INVALID
    assert read(k=None, tokens=3) == INVALID
    assert read(slots=None, tokens=3) == INVALID


def norm(qp=X, qs=256, qw=None, qo=Y, qos=256, hq=2, kp=Z, ks=128, kw=None, ko=W, kos=128, hk=1, d=128, tab=T, mp=9,
         rot=128, inter=0, pos=SL, eps=1e-6, tokens=0):
    return q.lib().nvfp4_qk_norm_rope(qp, qs, qw, qo, qos, hq, kp, ks, kw, ko, kos, hk, d, tab, mp, rot, inter, pos, eps,
                                      tokens, None)


def test_norm_rope_refusals():
    assert norm() == OK
    assert norm(tab=None, pos=None, rot=0) == OK
    assert norm(d=96) == UNSUP
    assert norm(rot=136) == SHAPE and norm(rot=12) == SHAPE and norm(rot=-8) == INVALID
    assert norm(tab=None) == INVALID and "cos_sin" in err()
    assert norm(pos=None) == INVALID and "positions" in err()
    assert norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID
    assert norm(hq=0) == UNSUP and norm(hk=0) == UNSUP
    assert norm(qs=128) == SHAPE
    assert norm(qs=260) == ALIGN
    assert norm(qw=P(0x18)) == ALIGN
    assert norm(tokens=1 << 30) == UNSUP
    for kw in (dict(qo=Z), dict(ko=X), dict(ko=Y), dict(qo=T), dict(ko=SL), dict(qo=P(X.value + 256))):
        assert norm(tokens=3, **kw) == INVALID and "overlap" in err(), kw
    # k's rows inside q's token stride share nothing; one value further they do
    assert norm(qs=384, qo=X, qos=384, kp=P(X.value + 512), ks=384, ko=P(X.value + 496), kos=384, tokens=3) == INVALID


def test_norm_rope_write_refusals():
    def f(c=None, qs=256, qo=Y, hq=2, kp=Z, vp=W, slots=SL, tokens=3, rot=128):
        return q.lib().nvfp4_qk_norm_rope_write(c or cache(heads=1), X, qs, None, qo, 256, hq, kp, 128, None, vp, 128, T, 9,
                                                rot, 0, P(0x50), 1e-6, slots, tokens, None)
    assert f(tokens=0) == OK
    assert f(cache(heads=1, ps=17)) == SHAPE
    assert f(vp=None) == INVALID and f(slots=None) == INVALID
    assert f(qo=KC) == INVALID and "overlap" in err()
    assert f(vp=VC) == INVALID and "overlap" in err()
    assert f(qo=W) == INVALID and "overlap" in err()
    assert f(rot=130) == SHAPE


def att(c=None, qp=X, qs=512, hq=4, starts=None, batch=3, total=3, mq=1, table=T, width=8, lens=Z, mkv=100, pre=None,
        plen=0, scale=0.1, out=Y, ws=W, wsn=1 << 26):
    return q.lib().nvfp4_kv_attention(c or cache(), qp, qs, hq, starts, batch, total, mq, table, width, lens, mkv, pre,
                                      plen, scale, out, ws, wsn, None)


def test_attention_refusals():
    empty = dict(batch=0, total=0)
    assert att(**empty) == OK
    assert att(hq=3) == SHAPE and "q_heads" in err()
    assert att(hq=0) == SHAPE
    assert att(qp=None) == INVALID and att(qs=256) == SHAPE and att(qs=514) == ALIGN
    assert att(lens=None) == INVALID and att(out=None) == INVALID
    assert att(table=None) == INVALID
    assert att(mkv=129) == SHAPE and "page table" in err()
    assert att(plen=5) == INVALID and "prefix_pages" in err()
    assert att(plen=-1) == INVALID
    assert att(mkv=0, width=0, plen=(1 << 31) - 1, pre=SL, mq=0) == INVALID
    assert att(width=1 << 28, mkv=1 << 30, pre=SL, plen=1 << 30) == UNSUP
    assert att(total=4) == INVALID and "q_starts" in err()
    assert att(mq=2) == INVALID and "q_starts" in err()
    assert att(batch=0) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert att(scale=s) == INVALID and "scale" in err()
    assert att(out=X) == INVALID and "overlap" in err()
    assert att(out=KC) == INVALID and "overlap" in err()
    assert att(out=Z) == INVALID and "overlap" in err()


def test_attention_workspace():
    lib = q.lib()

    def f(c=None, hq=4, batch=3, total=3, mq=1, mkv=100, plen=0):
        return lib.nvfp4_kv_attention_workspace_bytes(c or cache(), hq, batch, total, mq, mkv, plen)
    assert f(cache(ps=17)) == 0 and f(hq=3) == 0 and f(batch=-1) == 0
    n = f(mkv=100000, plen=3000)
    if n:
        big = dict(width=1 << 20, mkv=100000, pre=SL, plen=3000)
        assert att(ws=None, wsn=0, **big) == INVALID and "workspace" in err()
        assert att(wsn=n - 1, **big) == INVALID and "workspace" in err()
        assert att(ws=P(W.value + 16), wsn=n, **big) == ALIGN
        assert att(ws=X, wsn=n, **big) == INVALID and "overlap" in err()


def test_binding_refuses():
    import torch
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        q.KVCache(*(torch.zeros((1, 1, 16, 64), dtype=torch.uint8) for _ in range(6)))
    with pytest.raises(ValueError):
        q.nvfp4_qk_norm_rope(torch.zeros((2, 2, 64), dtype=bf), torch.zeros((2, 2, 64), dtype=bf), None, None, None, None)
    with pytest.raises(ValueError):
        q.nvfp4_qk_norm_rope(torch.zeros((2, 64), dtype=bf), torch.zeros((2, 64), dtype=bf), None, None, None, None)


def test_cache_is_fixed(monkeypatch):
    """The description that calls pass holds the addresses and sizes the cache
    was made with, so none of them can be exchanged under it."""
    import torch
    monkeypatch.setattr(q, "_need", lambda *a: None)                  # tensors of the host serve here
    u8 = torch.uint8
    parts = dict(k_codes=torch.zeros((2, 3, 32, 64), dtype=u8), k_scales=torch.zeros((2, 3, 32, 8), dtype=u8),
                 v_codes=torch.zeros((2, 3, 2, 64, 16), dtype=u8), v_scales=torch.zeros((2, 3, 2, 8, 16), dtype=u8),
                 k_gscale=torch.ones(1), v_gscale=torch.ones(1))
    c = q.KVCache(*parts.values())
    for name, t in parts.items():
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, t.clone())
        with pytest.raises(AttributeError, match=name):
            delattr(c, name)
        assert getattr(c, name) is t and getattr(c._struct, name) == t.data_ptr()
    for name, n in (("num_pages", 2), ("page_size", 32), ("kv_heads", 3), ("head_dim", 128)):
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, n + 1)
        assert getattr(c, name) == n == getattr(c._struct, name)
    with pytest.raises(AttributeError):
        c.device = "cuda:1"
    c.k_gscale.fill_(0.5)                                             # in place is how a scale is set
    assert copy.copy(c).k_codes is c.k_codes
    d = copy.deepcopy(c)
    assert d._struct.k_codes == d.k_codes.data_ptr() != c.k_codes.data_ptr() and d.k_gscale.item() == 0.5


def test_attention_refuses_more_queries_than_max_q_len_allows():
    """Rows past max_q_len of their sequence would be left as they were."""
    P_STARTS = P(0x20)
    assert att(starts=P_STARTS, total=4, mq=1) == INVALID and "max_q_len" in err()
    assert att(starts=P_STARTS, total=4000, batch=3, mq=1333) == INVALID and "max_q_len" in err()
    assert att(starts=P_STARTS, total=4000, batch=3, mq=1334, ws=None, wsn=0, mkv=129) == SHAPE      # the next check
    assert q.lib().nvfp4_kv_attention_workspace_bytes(cache(), 4, 3, 4000, 1333, 100000, 0) == 0


@pytest.mark.parametrize("given,want", [({}, 7), (dict(max_q_len=5), 5), (dict(q_starts=None), 1)])
def test_binding_takes_a_bound_that_always_holds(monkeypatch, given, want):
    """Without max_q_len, any one sequence may hold every query."""
    import torch
    seen = []

    class Lib:
        def nvfp4_kv_attention_workspace_bytes(self, ref, hq, batch, total, max_q_len, *rest):
            seen.append(max_q_len)
            return 0

        def nvfp4_kv_attention(self, ref, qp, qs, hq, starts, batch, total, max_q_len, *rest):
            seen.append(max_q_len)
            return 0

    class Cache:
        _index, head_dim, page_size, num_pages, kv_heads, _ref, device = -1, 64, 16, 4, 2, 0, "cpu"

    monkeypatch.setattr(q, "lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(q, "_attention_workspace", lambda *a: Lib().nvfp4_kv_attention_workspace_bytes(0, *a[5:]))
    batch = 7 if "q_starts" in given else 3
    args = dict(q_starts=torch.tensor([0, 0, 7, 7], dtype=torch.int32))
    args.update(given)
    q.nvfp4_kv_attention(torch.zeros((7, 4, 64), dtype=torch.bfloat16), Cache, torch.zeros((batch, 2), dtype=torch.int32),
                         torch.zeros(batch, dtype=torch.int32), **args)
    assert seen == [want, want]


def test_attention_bound_far_past_the_queries():
    """No sequence has more queries than there are rows: a larger max_q_len
    asks for no more than total_q does (its row tiles would not fit an int)."""
    def f(mq, hq=4, heads=2, total=300, **kw):
        a = dict(mkv=100000, plen=0)
        a.update(kw)
        return q.lib().nvfp4_kv_attention_workspace_bytes(cache(heads=heads), hq, 3, total, mq, a["mkv"], a["plen"])
    for kw in ({}, dict(plen=5000), dict(hq=128, heads=1, plen=70), dict(total=3)):
        want = f(kw.get("total", 300), **kw)
        assert want > 0, kw
        for mq in (301, 5000, (1 << 31) - 1):
            assert f(mq, **kw) == want, (kw, mq)
    big = dict(width=1 << 20, mkv=100000, starts=P(0x20), total=300, mq=(1 << 31) - 1)
    assert att(ws=None, wsn=0, **big) == INVALID and "workspace" in err()


def test_no_tokens_need_no_pointers():
    """An empty tensor's address is null: calls of no tokens do nothing."""
    assert write(k=None, v=None, slots=None, tokens=0) == OK
    assert read(slots=None, k=None, v=None, tokens=0) == OK
    assert norm(qp=None, qo=None, kp=None, ko=None, tokens=0) == OK
    lib = q.lib()
    assert lib.nvfp4_qk_norm_rope_write(cache(heads=1), None, 256, None, None, 256, 2, None, 128, None, None, 128, T, 9, 128,
                                        0, SL, 1e-6, None, 0, None) == OK
    assert att(qp=None, out=None, table=None, lens=None, batch=0, total=0) == OK
    assert att(qp=None, out=None, starts=P(0x20), total=0) == OK
    # what else is wrong with them is still said
    assert write(k=None, v=None, slots=None, ks=248, tokens=0) == SHAPE
    assert norm(qp=None, qo=None, kp=None, ko=None, rot=12) == SHAPE


def test_stride_of_a_single_token_does_not_matter():
    """A slice of one row keeps its buffer's pitch, whatever that is."""
    import torch
    buf = torch.zeros(2 * 300, dtype=torch.bfloat16)
    one = torch.as_strided(buf, (1, 2, 128), (300, 128, 1))
    assert q._rows(one, 2, 128, "k", -1) == (1, 2, 256)
    assert q._rows(one[:0], 2, 128, "k", -1) == (0, 2, 256)
    assert q._rows(torch.as_strided(buf, (2, 2, 128), (300, 128, 1)), 2, 128, "k", -1) == (2, 2, 300)


def test_launches_run_with_the_operands_device_current(monkeypatch):
    """A null stream is the current device's: a call on another device's
    tensors makes that device current for the launch, and only for it."""
    import torch
    q.lib()
    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i)
    monkeypatch.setattr(torch.cuda, "device", Device)
    seen = []

    def entry(*args):
        seen.append((now[0],) + args)
        return status

    status = OK
    for index in (0, 3):
        q._launch(index, entry, "a", 7)
        assert seen.pop() == (index, "a", 7, 100 + index) and now == [0]
    status = SHAPE
    with pytest.raises(q.Nvfp4Error):
        q._launch(3, entry)
    assert now == [0]
    # every function of the binding goes that way
    import inspect
    source = inspect.getsource(q)
    for name in q.SIGNATURES:
        if f"lib().{name}(" in source:
            assert name.endswith(("_bytes", "_slots", "last_error")), name


def test_calls_past_a_grid_are_refused_before_anything_runs():
    """A grid holds fewer than 2^32 threads: 64 a row for the join, 256 or 512
    for a segment."""
    f = q.lib().nvfp4_kv_attention_workspace_bytes
    one = cache(heads=1, d=64)
    rows = 1 << 20
    assert f(one, 63, rows, rows, 1, 16, 16) > 0
    big = dict(c=one, qs=64 * 64, hq=64, batch=rows, total=rows, table=T, width=1, mkv=16, pre=SL, plen=16)
    assert f(one, 64, rows, rows, 1, 16, 16) == 0
    assert att(**big) == UNSUP and "too large" in err()
    # segments: 2^24 workgroups of 256 threads, without partial results
    many = cache(heads=16, d=64)
    assert att(c=many, qs=16 * 64, hq=16, batch=rows, total=rows, width=1, mkv=16) == UNSUP and "too large" in err()
