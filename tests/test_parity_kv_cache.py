"""GPU parity of the cache operators: the quantizing write, the read back, the
head norms with rotation, and their one-launch form.

Codes, scales and values read back are compared bit for bit.  The head norms
are compared with the 64-bit formula: the kernel's sum of squares, root and
products cost a few ulps of fp32 (under 2^-20 of the two products a rotated
value is made of), and the one rounding to bf16 half an ulp (2^-8 of a value
just above a power of two)."""
import numpy as np
import pytest

import workloads
from oracle import formats as F
from oracle import kv as KV
from tests.gpu_util import Guarded, dev_bf16, host_bits, host_u8, log, need_gpu

pytestmark = pytest.mark.gpu

KG, VG = 0.013, 0.0071


def make_cache(torch, q, pages, ps, h, d, fill=0xA5):
    c = q.nvfp4_kv_cache(pages, ps, h, d, KG, VG)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(fill)
    return c


def expect_pages(bits, slots, pages, ps, h, d, g, transposed, fill=0xA5):
    codes, scales = KV.quantize_rows(bits, np.float32(g))
    rc = np.full((pages * ps, h, d // 2), fill, np.uint8)
    rs = np.full((pages * ps, h, d // 16), fill, np.uint8)
    for t, s in enumerate(slots):
        if 0 <= s < pages * ps:
            rc[s], rs[s] = codes[t], scales[t]
    return KV.to_pages(rc, ps, transposed), KV.to_pages(rs, ps, transposed), rc, rs


def pick_slots(rng, kind, tokens, total):
    if kind == "run":                                   # consecutive, unaligned start
        return np.arange(3, 3 + tokens)
    if kind == "aligned":
        return np.arange(16, 16 + tokens)
    s = rng.permutation(total)[:tokens]
    if kind == "padding":
        s = s.astype(np.int64)
        s[::3] = -1
        s[1::7] = total                                  # one past the end
        s[2::11] = 1 << 40
    return s


@pytest.mark.parametrize("tokens,h,d,ps,kind", [
    (1, 1, 64, 16, "run"), (1, 16, 128, 64, "shuffled"), (16, 2, 128, 16, "aligned"), (17, 3, 256, 32, "run"),
    (33, 2, 64, 16, "padding"), (100, 8, 128, 64, "padding"), (333, 4, 128, 128, "aligned"), (250, 1, 256, 16, "shuffled"),
    (64, 5, 64, 4096, "run"), (515, 2, 128, 16, "run"),
])
def test_write_and_read_bits(tokens, h, d, ps, kind):
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"kv write {tokens}x{h}x{d} ps={ps} {kind}")
    pages = (tokens + 40) // ps + 2
    rng = np.random.default_rng([7, tokens, h, d])
    slots = pick_slots(rng, kind, tokens, pages * ps)
    # rows of a packed projection, with outliers and exact zeros
    packed = workloads.random_bf16(720 + tokens, (tokens, 3 * h * d), outlier_frac=0.01, outlier_mul=25.0, zero_frac=0.05)
    packed[0, :h * d] = 0                                              # an all-zero K row
    dev = dev_bf16(packed)
    k = dev[:, :h * d].view(tokens, h, d)
    v = dev[:, 2 * h * d:].view(tokens, h, d)
    cache = make_cache(torch, q, pages, ps, h, d)
    st = torch.tensor(slots, dtype=torch.int64, device="cuda")
    q.nvfp4_kv_write(k, v, cache, st)
    ko, vo = Guarded((tokens, h, d), torch.bfloat16), Guarded((tokens, h, d), torch.bfloat16)
    q.nvfp4_kv_read(cache, st, out=(ko.t, vo.t))
    torch.cuda.synchronize()
    kb = packed[:, :h * d].reshape(tokens, h, d)
    vb = packed[:, 2 * h * d:].reshape(tokens, h, d)
    for bits, g, tr, codes, scales, out, name in ((kb, KG, False, cache.k_codes, cache.k_scales, ko, "K"),
                                                  (vb, VG, True, cache.v_codes, cache.v_scales, vo, "V")):
        wc, wsc, rc, rs = expect_pages(bits, slots, pages, ps, h, d, g, tr)
        assert np.array_equal(host_u8(codes), wc), f"{name} codes"
        assert np.array_equal(host_u8(scales), wsc), f"{name} scales"
        live = (slots >= 0) & (slots < pages * ps)
        want = np.zeros((tokens, h, d), np.uint16)
        dq = (F.e4m3_decode(rs[slots[live]].reshape(-1, d // 16)).astype(np.float32) * np.float32(g)).astype(np.float32)
        vals = F.e2m1_decode(np.stack((rc & 15, rc >> 4), -1).reshape(rc.shape[0], h, d))[slots[live]].reshape(-1, d)
        x = (vals.astype(np.float32) * np.repeat(dq, 16, axis=1)).astype(np.float32)
        want[live] = F.bf16_bits(F.bf16_round(x)).reshape(-1, h, d)
        got = host_bits(out.t)
        assert np.array_equal(got, want), f"{name} read back"
        assert out.intact()


def test_write_and_read_past_32_bits():
    """Pages whose codes lie beyond 4 GiB of the cache's base."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    h, d, ps, pages = 8, 256, 4096, 1100
    assert pages * ps * h * d // 2 > 1 << 32
    cache = q.nvfp4_kv_cache(pages, ps, h, d, KG, VG)
    tokens = 50
    slots = np.concatenate((np.arange(tokens - 10) + pages * ps - tokens, np.arange(10)))
    kb = workloads.random_bf16(741, (tokens, h * d)).reshape(tokens, h, d)
    vb = workloads.random_bf16(742, (tokens, h * d)).reshape(tokens, h, d)
    st = torch.tensor(slots, dtype=torch.int64, device="cuda")
    log("kv write past 4 GiB")
    q.nvfp4_kv_write(dev_bf16(kb), dev_bf16(vb), cache, st)
    ko, vo = q.nvfp4_kv_read(cache, st)
    torch.cuda.synchronize()
    for bits, g, got, codes, tr in ((kb, KG, ko, cache.k_codes, False), (vb, VG, vo, cache.v_codes, True)):
        wc, ws = KV.quantize_rows(bits, np.float32(g))
        for t in (0, 25, tokens - 10, tokens - 1):
            s = int(slots[t])
            row = codes[s // ps, :, s % ps] if not tr else codes[s // ps, :, (s % ps) // 16, :, s % 16]
            assert np.array_equal(host_u8(row), wc[t])
        assert np.allclose(F.bf16_from_bits(host_bits(got)), KV.values(wc, ws, np.float32(g)), rtol=2.0 ** -8, atol=0)


def check_norm(got_bits, x_bits, w_bits, table, pos, eps, rot, inter):
    want, mag = KV.norm_rope(F.bf16_from_bits(x_bits).astype(np.float64),
                             None if w_bits is None else F.bf16_from_bits(w_bits).astype(np.float64),
                             table.astype(np.float64), pos, eps, rot, inter)
    got = F.bf16_from_bits(got_bits).astype(np.float64)
    tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -20 * mag + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / tol):.2f} tol"


@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,weighted,strided", [
    (1, 1, 1, 64, 64, False, True, False), (1, 32, 16, 128, 128, False, True, True), (7, 64, 8, 128, 128, True, True, True),
    (33, 16, 4, 256, 256, False, True, False), (19, 12, 4, 64, 32, False, True, True), (5, 3, 3, 128, 8, False, False, True),
    (40, 8, 1, 128, 40, True, True, True), (21, 5, 1, 256, 0, False, True, True), (301, 64, 8, 128, 64, False, True, True),
])
def test_norm_rope(tokens, hq, hk, d, rot, inter, weighted, strided):
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"norm_rope {tokens}x{hq}+{hk}x{d} rot={rot} inter={inter}")
    rng = np.random.default_rng([11, tokens, d])
    total = (hq + 2 * hk) * d
    bits = workloads.random_bf16(760 + tokens, (tokens, total), sigma=3.0, outlier_frac=0.01, outlier_mul=40.0)
    bits[-1, :d] = 0                                                   # a head of zeros: eps keeps it finite
    dev = dev_bf16(bits)
    xq, xk = dev[:, :hq * d].view(tokens, hq, d), dev[:, hq * d:(hq + hk) * d].view(tokens, hk, d)
    if not strided:
        xq, xk = xq.contiguous(), xk.contiguous()
    wq = workloads.random_bf16(770, (1, d), sigma=1.0)[0] if weighted else None
    wk = workloads.random_bf16(771, (1, d), sigma=1.0)[0] if weighted else None
    ang = rng.uniform(-3, 3, (97, rot // 2))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    pos = rng.integers(0, 97, tokens)
    args = (dev_bf16(wq) if weighted else None, dev_bf16(wk) if weighted else None,
            torch.tensor(table, device="cuda") if rot else None,
            torch.tensor(pos, dtype=torch.int32, device="cuda") if rot else None)
    oq, ok = Guarded((tokens, hq, d), torch.bfloat16), Guarded((tokens, hk, d), torch.bfloat16)
    q.nvfp4_qk_norm_rope(xq, xk, *args, eps=1e-5, interleaved=inter, out=(oq.t, ok.t))
    torch.cuda.synchronize()
    check_norm(host_bits(oq.t), bits[:, :hq * d].reshape(tokens, hq, d), wq, table, pos, 1e-5, rot, inter)
    check_norm(host_bits(ok.t), bits[:, hq * d:(hq + hk) * d].reshape(tokens, hk, d), wk, table, pos, 1e-5, rot, inter)
    assert oq.intact() and ok.intact()

    # the one-launch form: the same q, and the cache bytes of the two calls
    ps = 16
    pages = tokens // ps + 3
    slots = rng.permutation(pages * ps)[:tokens]
    slots[::5] = -1
    st = torch.tensor(slots, dtype=torch.int64, device="cuda")
    v = dev[:, (hq + hk) * d:].view(tokens, hk, d)
    two, one = make_cache(torch, q, pages, ps, hk, d), make_cache(torch, q, pages, ps, hk, d)
    q.nvfp4_kv_write(ok.t, v, two, st)
    fused = q.nvfp4_qk_norm_rope_write(xq, xk, v, *args, one, st, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(fused.view(torch.int16), oq.t.view(torch.int16))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name

    # in place, inside the packed projection
    q.nvfp4_qk_norm_rope(xq, xk, *args, eps=1e-5, interleaved=inter, out=(xq, xk))
    torch.cuda.synchronize()
    assert torch.equal(xq.contiguous().view(torch.int16), oq.t.view(torch.int16))
    assert torch.equal(xk.contiguous().view(torch.int16), ok.t.view(torch.int16))
    if strided:
        assert np.array_equal(host_bits(dev[:, (hq + hk) * d:].contiguous()), bits[:, (hq + hk) * d:])


def test_position_outside_the_table_is_nan():
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    x = dev_bf16(workloads.random_bf16(790, (3, 128))).view(3, 1, 128)
    table = torch.cat((torch.ones(10, 32), torch.zeros(10, 32)), 1).cuda()
    log("norm_rope positions outside the table")
    yq, yk = q.nvfp4_qk_norm_rope(x, x.clone(), None, None, table,
                                  torch.tensor([-1, 10, 9], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for y in (yq, yk):
        n = torch.isnan(y[:, 0]).cpu()
        assert n[:2, :64].all() and not n[:2, 64:].any() and not n[2].any()


def test_another_stream():
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log("cache operators on another stream")
    bits = workloads.random_bf16(795, (64, 2 * 128))
    x = dev_bf16(bits).view(64, 2, 128)
    st = torch.arange(64, dtype=torch.int64, device="cuda")
    cache = make_cache(torch, q, 4, 16, 2, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x * 1.0                                    # made on this stream, used on it
        q.nvfp4_kv_write(y, y, cache, st)
        k, v = q.nvfp4_kv_read(cache, st)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want, _, _, _ = expect_pages(bits.reshape(64, 2, 128), np.arange(64), 4, 16, 2, 128, KG, False)
    assert np.array_equal(host_u8(cache.k_codes), want)
    assert torch.isfinite(k.float()).all() and torch.isfinite(v.float()).all()


def test_no_tokens():
    """Empty tensors go through every operator."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log("cache operators on no tokens")
    cache = make_cache(torch, q, 2, 16, 2, 128)
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    i32, i64 = (torch.empty(0, dtype=t, device="cuda") for t in (torch.int32, torch.int64))
    table = torch.ones((9, 128), device="cuda")
    q.nvfp4_kv_write(none, none, cache, i64)
    outs = [*q.nvfp4_kv_read(cache, i64), *q.nvfp4_qk_norm_rope(none, none, None, None, table, i32),
            q.nvfp4_qk_norm_rope_write(none, none, none, None, None, table, i32, cache, i64),
            q.nvfp4_kv_attention(none, cache, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), i32),
            q.nvfp4_kv_attention(none, cache, torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
                                 torch.zeros(2, dtype=torch.int32, device="cuda"),
                                 q_starts=torch.zeros(3, dtype=torch.int32, device="cuda"))]
    torch.cuda.synchronize()
    assert all(o.shape == (0, 2, 128) for o in outs)
    assert (host_u8(cache.k_codes) == 0xA5).all() and (host_u8(cache.v_scales) == 0xA5).all()


def test_one_token_of_an_odd_pitch():
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log("cache operators on one token of a row of 261 values")
    buf = dev_bf16(workloads.random_bf16(797, (1, 261)))
    x = torch.as_strided(buf, (1, 2, 128), (261, 128, 1))
    whole = x.clone(memory_format=torch.contiguous_format)
    st = torch.tensor([5], dtype=torch.int64, device="cuda")
    a, b = make_cache(torch, q, 1, 16, 2, 128), make_cache(torch, q, 1, 16, 2, 128)
    q.nvfp4_kv_write(x, x, a, st)
    q.nvfp4_kv_write(whole, whole, b, st)
    ya = q.nvfp4_qk_norm_rope(x, x, None, None, None, None)
    yb = q.nvfp4_qk_norm_rope(whole, whole, None, None, None, None)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([6], dtype=torch.int32, device="cuda")
    oa, ob = (q.nvfp4_kv_attention(t, a, table, lens) for t in (x, whole))
    torch.cuda.synchronize()
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    for u, w in ((ya[0], yb[0]), (ya[1], yb[1]), (oa, ob)):
        assert torch.equal(u.view(torch.int16), w.view(torch.int16))
    q.nvfp4_qk_norm_rope(x, x.clone(), None, None, None, None, out=(x, whole))            # in place
    torch.cuda.synchronize()
    assert torch.equal(x.contiguous().view(torch.int16), yb[0].view(torch.int16))


@pytest.mark.parametrize("sigma,eps", [(2.0 ** -64, 0.0), (2.0 ** -64, 1e-42), (2.0 ** -70, 1e-39), (2.0 ** -62, 1e-38)])
def test_norm_of_rows_whose_squares_are_denormal(sigma, eps):
    """The mean square is below the smallest normal float; its root is not."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log(f"norm_rope sigma {sigma} eps {eps}")
    rng = np.random.default_rng(23)
    bits = workloads.random_bf16(798, (20, 4 * 128), sigma=sigma)
    if eps > 0:
        bits[3, :128] = 0
    x = dev_bf16(bits).view(20, 4, 128)
    ang = rng.uniform(-3, 3, (9, 64))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    pos = rng.integers(0, 9, 20)
    eps = float(np.float32(eps))
    yq, yk = q.nvfp4_qk_norm_rope(x[:, :3], x[:, 3:], None, None, torch.tensor(table, device="cuda"),
                                  torch.tensor(pos, dtype=torch.int32, device="cuda"), eps=eps)
    torch.cuda.synchronize()
    check_norm(host_bits(yq), bits.reshape(20, 4, 128)[:, :3], None, table, pos, eps, 128, False)
    check_norm(host_bits(yk), bits.reshape(20, 4, 128)[:, 3:], None, table, pos, eps, 128, False)


def test_infinities_keep_their_sign():
    """code = sign(x) | E2M1(|x| / d) holds for infinities too, under a given
    global scale, in nvfp4_quantize and in the write."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log("infinities under a given scale")
    h, d = 2, 64
    bits = workloads.random_bf16(821, (5, h * d))
    for t, at, x in ((0, 3, np.inf), (1, 20, -np.inf), (2, 64, -np.inf), (2, 67, np.inf), (4, 127, -np.inf)):
        bits[t, at] = F.bf16_bits(np.array([x], np.float32))[0]
    for g in (KG, 2.0 ** -70):                           # quotients from reciprocals, and divided
        wc, ws = KV.quantize_rows(bits.reshape(5, h, d), np.float32(g))
        c, s, _ = q.nvfp4_quantize(dev_bf16(bits).view(5 * h, d), global_scale=torch.full((1,), g, device="cuda"))
        cache = q.nvfp4_kv_cache(1, 16, h, d, g, g)
        q.nvfp4_kv_write(dev_bf16(bits).view(5, h, d), dev_bf16(bits).view(5, h, d), cache, torch.arange(5, device="cuda"))
        torch.cuda.synchronize()
        assert np.array_equal(host_u8(c).reshape(wc.shape), wc) and np.array_equal(host_u8(s).reshape(ws.shape), ws)
        for pages, want, frag in ((cache.k_codes, wc, False), (cache.k_scales, ws, False),
                                  (cache.v_codes, wc, True), (cache.v_scales, ws, True)):
            assert np.array_equal(np.stack([KV.rows_at(host_u8(pages), t, frag) for t in range(5)]), want)


def test_infinities_and_nan_are_stored_finite():
    """As nvfp4_quantize stores them, in every form of the write; and a query
    that does not see such a token has the same output as without it."""
    torch = need_gpu()
    import quantized_gemm_nvfp4_amd as q
    log("infinities and NaN into the cache")
    tokens, h, d = 40, 2, 128
    k = dev_bf16(workloads.random_bf16(811, (tokens, h * d))).view(tokens, h, d)
    v = dev_bf16(workloads.random_bf16(812, (tokens, h * d))).view(tokens, h, d)
    bad_k, bad_v = k.clone(), v.clone()
    for t, x in ((30, float("nan")), (31, float("inf")), (32, -float("inf")), (33, -float("nan"))):
        bad_k[t, 0, t] = bad_v[t, 1, 2 * t] = x
    slots = torch.arange(tokens, device="cuda") + 5
    caches = []
    for a, b in ((k, v), (bad_k, bad_v)):
        c = make_cache(torch, q, 3, 16, h, d)
        q.nvfp4_kv_write(a, b, c, slots)
        caches.append(c)
    clean, bad = caches
    back = q.nvfp4_kv_read(bad, slots)
    for rows, g, got, pages, frag in ((bad_k, bad.k_gscale, back[0], (bad.k_codes, bad.k_scales), False),
                                      (bad_v, bad.v_gscale, back[1], (bad.v_codes, bad.v_scales), True)):
        codes, scales, _ = q.nvfp4_quantize(rows.view(tokens * h, d), global_scale=g)
        for want, have in zip((codes, scales), pages):
            plain = np.stack([KV.rows_at(host_u8(have), s, frag) for s in slots.tolist()])
            assert np.array_equal(plain, host_u8(want).reshape(plain.shape))
        assert torch.isfinite(got.float()).all()
        odd = ~torch.isfinite(rows)
        top = torch.full_like(got.float(), 1.0) * 6 * 448 * g
        assert torch.equal(got[odd].float().abs(), top.bfloat16()[odd].float())
        keep = odd & ~torch.isnan(rows)
        assert torch.equal(got[keep] > 0, rows[keep] > 0)
    # queries 0 .. 39 of one sequence whose keys are all 40 tokens: 0 .. 29 see none of the four
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([tokens + 5], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    first = torch.arange(5, device="cuda")                              # the slots in front
    for c in caches:
        q.nvfp4_kv_write(k[:5], v[:5], c, first)
    qs = dev_bf16(workloads.random_bf16(813, (tokens, 8 * d))).view(tokens, 8, d)
    a, b = (q.nvfp4_kv_attention(qs, c, table, lens, q_starts=starts, max_q_len=tokens) for c in caches)
    torch.cuda.synchronize()
    assert torch.equal(a[:30].view(torch.int16), b[:30].view(torch.int16)) and torch.isfinite(b.float()).all()

    # a position outside the table, in the one-launch form
    cos_sin = torch.cat((torch.ones(10, 64), torch.zeros(10, 64)), 1).cuda()
    pos = torch.tensor([3, 10, -1, 9], dtype=torch.int32, device="cuda")
    one, two = make_cache(torch, q, 1, 16, h, d), make_cache(torch, q, 1, 16, h, d)
    st = torch.arange(4, device="cuda")
    yq = q.nvfp4_qk_norm_rope_write(qs[:4], k[:4], v[:4], None, None, cos_sin, pos, one, st)
    _, yk = q.nvfp4_qk_norm_rope(qs[:4], k[:4], None, None, cos_sin, pos)
    q.nvfp4_kv_write(yk, v[:4], two, st)
    rk, rv = q.nvfp4_kv_read(one, st)
    torch.cuda.synchronize()
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name
    nan = torch.isnan(yq).flatten(1).any(1).tolist()
    assert nan == [False, True, True, False] and torch.isfinite(rk.float()).all() and torch.isfinite(rv.float()).all()
