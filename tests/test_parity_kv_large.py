"""GPU parity of the cache operators at sizes where calls are laid out otherwise
than small ones: shares of many passes and more than 64 sequences in the
attention, several rows or pieces a thread in the other operators.

The reference is computed on the device from the cache's own bytes, in 64 bits
(attention) or as the format's fp32 steps (read), by this file's tables."""
import numpy as np
import pytest

import workloads
from oracle import formats as F
from tests.gpu_util import Guarded, dev_bf16, host_bits, log, need_gpu
from tests.test_parity_kv_cache import check_norm

pytestmark = pytest.mark.gpu

KG, VG = 0.013, 0.0071


def tables(torch, dtype):
    """Values of a packed byte's two codes and of an E4M3 byte (NaN included)."""
    c = np.arange(256, dtype=np.uint8)
    pairs = np.stack((F.e2m1_decode(c & 15), F.e2m1_decode(c >> 4)), 1)
    return (torch.tensor(pairs, dtype=dtype, device="cuda"),
            torch.tensor(F.e4m3_decode(c), dtype=dtype, device="cuda"))


def rows_of(torch, cache, which, slots, dtype):
    """K or V of every head at `slots`: values [tokens, heads, D] without g, and
    their block scales, repeated."""
    pairs, e4m3 = tables(torch, dtype)
    page, at = slots // cache.page_size, slots % cache.page_size
    if which == "k":
        c, s = cache.k_codes[page, :, at], cache.k_scales[page, :, at]
    else:
        c, s = cache.v_codes[page, :, at // 16, :, at % 16], cache.v_scales[page, :, at // 16, :, at % 16]
    return pairs[c.long()].flatten(-2), e4m3[s.long()].repeat_interleave(16, -1)


class Batch:
    """Sequences in shuffled pages of a cache of random rows (0xFF past the
    sequences' ends)."""

    def __init__(self, torch, q, hq, hkv, d, ps, lens, nq, prefix, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.ps, self.lens, self.nq, self.prefix = hq, hkv, d, ps, lens, nq, prefix
        need = [-(-n // ps) for n in [prefix] + lens]
        order = rng.permutation(sum(need) + 1).astype(np.int32)
        ends = np.cumsum([0] + need)
        own = [order[ends[i]:ends[i + 1]] for i in range(len(need))]
        table = np.full((len(lens), max(1, max(need[1:]))), -1, np.int32)
        for b, pages in enumerate(own[1:]):
            table[b, :len(pages)] = pages
        self.slots = [torch.tensor((p.astype(np.int64)[:, None] * ps + np.arange(ps)).reshape(-1)[:n], device="cuda")
                      for p, n in zip(own, [prefix] + lens)]
        self.table = torch.tensor(table, device="cuda")
        self.prefix_pages = torch.tensor(own[0], device="cuda") if prefix else None
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(np.cumsum([0] + nq), dtype=torch.int32, device="cuda")
        self.cache = q.nvfp4_kv_cache(len(order), ps, hkv, d, KG, VG)
        for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
            t.fill_(0xFF)
        channel = 1.0 + 5.0 * (torch.rand((hkv, d), generator=gen, device="cuda") > 0.98)
        for s in self.slots:
            k, v = (torch.randn((len(s), hkv, d), generator=gen, device="cuda") for _ in range(2))
            q.nvfp4_kv_write((k * channel).bfloat16(), v.bfloat16(), self.cache, s)
        self.q = (torch.randn((sum(nq), hq, d), generator=gen, device="cuda") * 1.5).bfloat16()

    def call(self, q, out, **kw):
        return q.nvfp4_kv_attention(self.q, self.cache, self.table, self.kv_lens, out=out, max_kv_len=max(self.lens),
                                    q_starts=None if self.nq == [1] * len(self.nq) else self.starts,
                                    max_q_len=max(self.nq), prefix_pages=self.prefix_pages, prefix_len=self.prefix, **kw)

    def check(self, torch, out):
        """The tolerance is that of test_parity_kv_attention.py."""
        f64, group, scale, at = torch.float64, self.hq // self.hkv, self.d ** -0.5, 0
        for b, (n, m) in enumerate(zip(self.lens, self.nq)):
            total = self.prefix + n
            if m == 0:
                continue
            if total == 0:
                assert not out[at:at + m].any(), f"sequence {b}"
                at += m
                continue
            s = torch.cat((self.slots[0], self.slots[1 + b]))
            k, v = (torch.mul(*rows_of(torch, self.cache, w, s, f64)) * float(np.float32(g)) for w, g in (("k", KG), ("v", VG)))
            last = total - m + torch.arange(m, device="cuda")
            hidden = (torch.arange(total, device="cuda")[None] > last[:, None]).repeat_interleave(group, 0)
            for h in range(self.hkv):
                x = self.q[at:at + m, h * group:(h + 1) * group].to(f64).reshape(m * group, self.d)
                kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
                p = torch.matmul(x, kh.T.contiguous()).mul_(scale).masked_fill_(hidden, -float("inf"))
                p = torch.exp(p - p.amax(1, keepdim=True).clamp(min=-1e300))
                norm = p.sum(1, keepdim=True)
                p = torch.where(norm > 0, p / norm, p)
                want, a = torch.matmul(p, vh), torch.matmul(p, vh.abs())
                big = torch.matmul(x.abs(), kh.abs().T.contiguous()).mul_(scale).masked_fill_(hidden, 0.0).amax(1, keepdim=True)
                tol = (2.0 ** -8 * want.abs() * (1 + 2.0 ** -7)
                       + a * (2.0 ** -11 + 2.0 ** -16 + 2 * (self.d + 8) * 2.0 ** -24 * big)
                       + 2.0 ** -32 * vh.abs().sum(0) + 1e-30)
                got = out[at:at + m, h * group:(h + 1) * group].to(f64).reshape(m * group, self.d)
                ratio = ((got - want).abs() / tol).nan_to_num(nan=1e9).max().item()
                assert ratio <= 1.0, f"sequence {b} ({n} keys, {m} queries), head {h}: {ratio:.2f} of the tolerance"
            at += m


def ragged(batch, hi, empty=()):
    rng = np.random.default_rng([batch, hi])
    lens = [int(x) for x in rng.integers(1, hi + 1, batch)]
    for i in empty:
        lens[i] = 0
    lens[batch // 2] = hi
    return lens


SHARES = [
    # hq, hkv, d, ps, lens, queries, prefix, rows of a streaming row tile
    (16, 2, 128, 64, ragged(70, 7000, (0, 63, 64, 65)), 1, 0, 16),
    (16, 4, 64, 16, ragged(130, 6000, (63, 64, 127, 128, 129)), 1, 0, 16),
    (8, 2, 256, 16, ragged(9, 20000, (3,)), 1, 0, 16),
    (8, 4, 128, 128, ragged(65, 2500, (64,)), 1, 300, 16),
    (12, 4, 256, 64, ragged(66, 1500, (0, 1, 2)), 1, 130, 16),
    (40, 2, 128, 64, ragged(24, 8000, (7,)), 1, 0, 32),                  # 20 rows a head
    (40, 2, 64, 32, ragged(24, 9000, (23,)), 1, 70, 32),
    (18, 1, 256, 16, ragged(20, 16000, (0,)), 1, 0, 32),
    (40, 1, 128, 64, ragged(68, 6000, (63, 64)), 1, 0, 32),              # 40 rows: two row tiles
    (8, 2, 128, 16, ragged(30, 8000, (11,)), 5, 0, 32),                  # 1 to 5 queries a sequence
    (8, 2, 128, 64, ragged(30, 8000, (12,)), 9, 200, 32),                # two row tiles, most of them half empty
    (4, 2, 256, 64, ragged(40, 7000, (39,)), 30, 0, 32),
]


@pytest.mark.parametrize("case", SHARES, ids=[f"{c[0]}h{c[1]}d{c[2]}p{c[3]}b{len(c[4])}q{c[5]}x{c[6]}" for c in SHARES])
def test_shares_of_many_passes(case):
    """Workers that take several passes each, go on from one sequence and row
    tile to the next, and leave partial results at both ends."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    hq, hkv, d, ps, lens, nq, prefix, tile = case
    log(f"kv attention in shares: {hq} on {hkv} heads of {d}, {len(lens)} sequences of up to {max(lens)}, {nq} queries, prefix {prefix}")
    rng = np.random.default_rng(5)
    queries = [1] * len(lens) if nq == 1 else [int(x) for x in rng.integers(1, nq + 1, len(lens))]
    if nq > 1:
        queries[0], queries[1] = nq, 0
    b = Batch(torch, q, hq, hkv, d, ps, lens, queries, prefix)
    # without a prefix the workspace is the workers' two slots of a row tile each
    parts = q.lib().nvfp4_kv_attention_workspace_bytes(b.cache._ref, hq, len(lens), sum(queries), max(queries), max(lens),
                                                       0) // (8 + 4 * d)
    workers = parts // (2 * tile)
    tiles = -(-max(queries) * (hq // hkv) // tile)
    total = sum(max(1, -(-n // 256)) for n in lens) * hkv * tiles
    assert parts % (2 * tile) == 0 and 0 < workers < total, (workers, total)
    out = Guarded((sum(queries), hq, d), torch.bfloat16)
    b.call(q, out.t)
    torch.cuda.synchronize()
    assert out.intact()
    b.check(torch, out.t)
    first = out.t.clone()
    b.call(q, out.t)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), out.t.view(torch.int16)), "two calls differ"


LARGE = [
    # hq, hkv, d, ps, lens, queries, prefix
    (32, 16, 128, 64, [12, 0], [11, 1], 16500),          # the prefix on two row tiles of 16
    (32, 16, 128, 16, [0, 40, 3], [5, 9, 1], 16500),
    (32, 16, 256, 64, [12, 0], [11, 1], 16500),
    (16, 8, 256, 32, [5, 70], [9, 7], 33100),
    (16, 2, 128, 64, ragged(130, 300, (63, 64, 65, 129)), [1] * 130, 0),         # more than 64 whole sequences
    (16, 2, 64, 16, ragged(200, 500, (0, 64, 128)), [2] * 64 + [0] * 3 + [1] * 133, 0),
    (8, 2, 128, 32, ragged(150, 200, (64,)), [1] * 150, 700),
    (8, 2, 128, 64, [9000, 300, 0, 64], [600, 1, 2, 64], 0),                     # chunks and single tokens
    (8, 2, 64, 64, [6000, 300, 1, 2000], [700, 1, 1, 130], 3000),
    (8, 2, 256, 64, [5000, 300, 1, 2000], [300, 1, 1, 130], 1000),
]


@pytest.mark.parametrize("case", LARGE, ids=[f"{c[0]}h{c[1]}d{c[2]}p{c[3]}b{len(c[4])}q{max(c[5])}x{c[6]}" for c in LARGE])
def test_large_calls(case):
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    hq, hkv, d, ps, lens, queries, prefix = case
    log(f"kv attention, large: {hq} on {hkv} heads of {d}, {len(lens)} sequences, {max(queries)} queries, prefix {prefix}")
    b = Batch(torch, q, hq, hkv, d, ps, lens, queries, prefix)
    out = Guarded((sum(queries), hq, d), torch.bfloat16)
    b.call(q, out.t)
    torch.cuda.synchronize()
    assert out.intact()
    b.check(torch, out.t)


@pytest.mark.parametrize("h,d,ps,tokens", [(5, 64, 16, 30005), (8, 128, 64, 9003), (3, 256, 32, 12007), (1, 64, 4096, 140001)])
def test_read_of_a_long_list(h, d, ps, tokens):
    """Runs that begin anywhere in a fragment, cross pages, are broken by
    padding, and scattered slots, in a list long enough for the wide kernel."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"kv read of {tokens} tokens, {h} heads of {d}, pages of {ps}")
    assert tokens * h * d // 8 >= 256 * 4 * 1024 and tokens % 16
    rng = np.random.default_rng([h, d])
    slots, at = [], 0
    while len(slots) < tokens:
        kind, n = rng.integers(0, 8), int(rng.integers(1, 90))
        at += int(rng.integers(0, 40))
        slots += range(at, at + n)
        at += n
        if kind == 0:
            slots += [-1] * int(rng.integers(1, 20))
        elif kind == 1:
            slots += [int(x) for x in rng.integers(0, at, int(rng.integers(1, 40)))]
    slots = np.array(slots[:tokens], np.int64)
    pages = at // ps + 1
    slots[rng.integers(0, tokens, 50)] = -1
    slots[rng.integers(0, tokens, 5)] = pages * ps                      # one past the end
    starts = slots[::16][:tokens // 16]
    runs = np.all(slots[:tokens // 16 * 16].reshape(-1, 16) == starts[:, None] + np.arange(16), 1) & (starts >= 0)
    assert len(set((starts[runs] % 16).tolist())) == 16 and not runs.all()          # every offset, and the other path
    cache = q.nvfp4_kv_cache(pages, ps, h, d, KG, VG)
    gen = torch.Generator(device="cuda").manual_seed(d)
    for t in (cache.k_codes, cache.v_codes):
        t.random_(0, 256, generator=gen)
    for t in (cache.k_scales, cache.v_scales):
        t.random_(0, 127, generator=gen)
    st = torch.tensor(slots, device="cuda")
    ko, vo = Guarded((tokens, h, d), torch.bfloat16), Guarded((tokens, h, d), torch.bfloat16)
    q.nvfp4_kv_read(cache, st, out=(ko.t, vo.t))
    torch.cuda.synchronize()
    assert ko.intact() and vo.intact()
    live = (st >= 0) & (st < pages * ps)
    for name, out, g in (("k", ko.t, KG), ("v", vo.t, VG)):
        value, scale = rows_of(torch, cache, name, st.clamp(0, pages * ps - 1), torch.float32)
        want = torch.where(live[:, None, None], value * (scale * np.float32(g).item()), torch.zeros(()).cuda()).bfloat16()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), name


@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,strided", [
    (8211, 13, 4, 64, 64, False, True), (8211, 13, 4, 64, 32, True, False), (16390, 6, 2, 64, 0, False, True),
    (3001, 32, 3, 128, 128, False, True), (2051, 31, 2, 128, 64, True, True), (66001, 1, 1, 128, 40, False, False),
    (2503, 11, 4, 256, 256, True, True), (1303, 24, 2, 256, 128, False, True),
])
def test_norm_of_many_tokens(tokens, hq, hk, d, rot, inter, strided):
    """Four rows a thread: the same bits as calls of a few tokens, in every
    form, and a sample against the formula."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"norm_rope of {tokens} tokens, {hq} + {hk} heads of {d}, rot {rot}")
    assert tokens * (hq + hk) * d >= 256 * 16 * 2048
    gen, rng = torch.Generator(device="cuda").manual_seed(tokens), np.random.default_rng(tokens)
    packed = (torch.randn((tokens, (hq + 2 * hk) * d), generator=gen, device="cuda") * 3).bfloat16()
    xq, xk, xv = (t.view(tokens, -1, d) for t in packed.split((hq * d, hk * d, hk * d), 1))
    if not strided:
        xq, xk, xv = xq.contiguous(), xk.contiguous(), xv.contiguous()
    ang = rng.uniform(-3, 3, (301, rot // 2))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    pos = rng.integers(0, 301, tokens)
    w = [workloads.random_bf16(830 + i, (1, d), sigma=1.0)[0] for i in range(2)]
    weights = [dev_bf16(x) for x in w]
    rotation = (torch.tensor(table, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda")) if rot else (None, None)
    oq, ok = Guarded((tokens, hq, d), torch.bfloat16), Guarded((tokens, hk, d), torch.bfloat16)
    q.nvfp4_qk_norm_rope(xq, xk, *weights, *rotation, eps=1e-5, interleaved=inter, out=(oq.t, ok.t))
    torch.cuda.synchronize()
    assert oq.intact() and ok.intact()
    step = 200
    for t in range(0, tokens, step):
        a, b = q.nvfp4_qk_norm_rope(xq[t:t + step], xk[t:t + step], *weights, rotation[0],
                                    rotation[1][t:t + step].clone() if rot else None, eps=1e-5, interleaved=inter)
        assert torch.equal(a.view(torch.int16), oq.t[t:t + step].view(torch.int16)), t
        assert torch.equal(b.view(torch.int16), ok.t[t:t + step].view(torch.int16)), t
    some = np.concatenate((np.arange(9), rng.integers(0, tokens, 60), np.arange(tokens - 9, tokens)))
    at = torch.tensor(some, device="cuda")
    for x, y, weight in ((xq, oq.t, w[0]), (xk, ok.t, w[1])):
        check_norm(host_bits(y[at]), host_bits(x[at].contiguous()), weight, table, pos[some], 1e-5, rot, inter)

    # with the cache: the same q, and the bytes of the two calls
    ps = 32
    pages = tokens // ps + 2
    slots = rng.permutation(pages * ps)[:tokens]
    slots[::7] = -1
    st = torch.tensor(slots, device="cuda")
    one, two = (q.nvfp4_kv_cache(pages, ps, hk, d, KG, VG) for _ in range(2))
    for c in (one, two):
        for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
            t.fill_(0xA5)
    q.nvfp4_kv_write(ok.t, xv, two, st)
    fused = Guarded((tokens, hq, d), torch.bfloat16)
    q.nvfp4_qk_norm_rope_write(xq, xk, xv, *weights, *rotation, one, st, eps=1e-5, interleaved=inter, out=fused.t)
    torch.cuda.synchronize()
    assert fused.intact() and torch.equal(fused.t.view(torch.int16), oq.t.view(torch.int16))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name


@pytest.mark.parametrize("h,d,ps,tokens", [(5, 64, 16, 20003), (8, 128, 64, 9001), (3, 256, 4096, 7009)])
def test_write_of_a_long_list(h, d, ps, tokens):
    """Every row as nvfp4_quantize has it, at its slot and nowhere else."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"kv write of {tokens} tokens, {h} heads of {d}, pages of {ps}")
    gen, rng = torch.Generator(device="cuda").manual_seed(tokens), np.random.default_rng(tokens)
    pages = tokens // ps + 2
    slots = np.roll(np.arange(pages * ps), 5)[:tokens].copy()
    cut = tokens // 3
    slots[:cut] = rng.permutation(slots[:cut])
    slots[rng.integers(0, tokens, 60)] = -1
    st = torch.tensor(slots, device="cuda")
    k, v = (torch.randn((tokens, h, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    cache = q.nvfp4_kv_cache(pages, ps, h, d, KG, VG)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    q.nvfp4_kv_write(k, v, cache, st)
    live = st >= 0
    for rows, g, codes, scales, frag in ((k, cache.k_gscale, cache.k_codes, cache.k_scales, False),
                                         (v, cache.v_gscale, cache.v_codes, cache.v_scales, True)):
        c, s, _ = q.nvfp4_quantize(rows.view(tokens * h, d), global_scale=g)
        for want, pool in ((c, codes), (s, scales)):
            # the pool as rows in slot order
            rows_in = (pool.permute(0, 2, 4, 1, 3) if frag else pool.permute(0, 2, 1, 3)).reshape(pages * ps, h, -1)
            expect = torch.full_like(rows_in, 0xA5)
            expect[st[live]] = want.view(tokens, h, -1)[live]
            assert torch.equal(rows_in, expect)
