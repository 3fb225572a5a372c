"""Block-scaled FP8 layer and mixture of experts on the GPU against plain 64-bit statements (fp8b_ref.py).

Tolerances, fixed before the first run:
  * codes, scales, ids, offsets and positions are equal;
  * a product's sum is within 2^-12 of the sum of its terms' magnitudes, the bound that the library's other
    E4M3 products are held to (the tensor core's accumulation inside a block is not fp32's), and Y adds half a
    bf16 step, 2^-8 of the value's power of two at most;
  * what follows from a product (h, its codes) carries that bound through the formulas.
"""
from __future__ import annotations

import pytest
import torch

import fp8b_ref as ref
import mixed_precision_gemm_b200 as sq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACC = 2.0 ** -12          # of the sum of magnitudes
HALF_BF16 = 2.0 ** -8     # of the value


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def activations(M, K, seed=0):
    g = gen(seed)
    x = torch.randn(M, K, device=DEV, generator=g)
    x[:, torch.randperm(K, device=DEV, generator=g)[:max(1, K // 64)]] *= 30.0
    return x.bfloat16()


def weights(*shape, seed=1):
    return (torch.randn(*shape, device=DEV, generator=gen(seed)) * shape[-1] ** -0.5).bfloat16()


def check_product(y, total, mags):
    """y bf16 against the 64-bit sum, with the bounds above."""
    err = (y.double() - total).abs()
    lim = ACC * mags + HALF_BF16 * (total.abs() + ACC * mags)
    assert bool((err <= lim).all()), f"worst {(err - lim).max().item():.3g} over the bound"


# ------------------------------------------------------------------ quantizers
@pytest.mark.parametrize("M,K", [(1, 8), (3, 128), (5, 136), (7, 1000), (130, 520), (33, 8192), (2, 65536)])
def test_quant_rows_bits(M, K):
    x = activations(M, K)
    x[0, : min(K, 128)] = 0                       # an empty block
    if M > 1:
        x[1, ::3] = -0.0
        x[1, : min(K, 128)] *= 2.0 ** -120        # scales below 2^-100
        x[-1, -8:] = torch.tensor([448, 1.0625, -1.0625, 2.0 ** -9, 2.0 ** -10, -(2.0 ** -10), 3 * 2.0 ** -10, 0.0],
                                  device=DEV).bfloat16()   # ties where the block's scale is 1
    if M > 2 and K >= 128:
        x[2, :128] = (torch.arange(128, device=DEV) % 9 * 9.2e-41).bfloat16()  # bf16 subnormals
    c, s = sq.quant_fp8b(x)
    rc, rs = ref.quant_rows(x)
    assert torch.equal(s, rs)
    assert torch.equal(c, rc)


def test_quant_strided_rows_and_every_bf16_value():
    bits = torch.arange(0, 0x7F80, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    for top in (448.0, 3.0e38, 1.0, 1.0e-3, 3.0e-39):
        v = torch.where(bits.float() <= top, bits.float(), torch.zeros_like(bits.float())).bfloat16()
        wide = torch.zeros(256, 160, dtype=torch.bfloat16, device=DEV)
        wide[:, 8:135] = torch.nn.functional.pad(v, (0, 256 * 127 - v.numel())).view(256, 127) * torch.tensor(
            [1.0, -1.0], device=DEV).repeat(64)[:127].bfloat16()
        wide[:, 135] = top
        x = wide[:, 8:136]
        c, s = sq.quant_fp8b(x)
        rc, rs = ref.quant_rows(x)
        assert torch.equal(s, rs) and torch.equal(c, rc), top


@pytest.mark.parametrize("shape", [(8, 8), (128, 128), (136, 264), (1000, 520), (3, 2, 200, 136)])
def test_prepare_weights_bits(shape):
    w = weights(*shape)
    w.view(-1, *shape[-2:])[0, :, : min(128, shape[-1])] = 0
    pw = sq.prepare_weights_fp8b(w)
    wc, ws = pw.W_8.view(-1, *pw.W_8.shape[-2:]), pw.s_w.view(-1, *pw.s_w.shape[-2:])
    for g, m in enumerate(w.view(-1, *shape[-2:])):
        rc, rs = ref.quant_weights(m)
        assert torch.equal(ws[g], rs) and torch.equal(wc[g], rc)


def test_prepare_weights_strided():
    w = weights(3, 264, 400)[:, 8:208, 8:272]
    pw = sq.prepare_weights_fp8b(w)
    for g in range(3):
        rc, rs = ref.quant_weights(w[g])
        assert torch.equal(pw.s_w[g], rs) and torch.equal(pw.W_8[g], rc)


# ------------------------------------------------------------------ one product
@pytest.mark.parametrize("M,K,N", [
    (1, 8, 8), (1, 128, 128), (1, 4096, 1048), (2, 136, 120), (7, 1000, 264), (15, 512, 512), (16, 640, 128),
    (17, 256, 1024), (33, 2048, 136), (64, 1032, 384), (65, 128, 2056), (100, 4104, 520), (128, 384, 256),
    (129, 384, 256), (192, 128, 8), (255, 520, 776), (256, 1024, 512), (257, 1152, 1032), (513, 2048, 640),
    (1000, 264, 2000), (2100, 896, 1280), (300, 8192, 264), (1, 65536, 8), (140, 16384, 136)])
def test_linear(M, K, N):
    x, w = activations(M, K), weights(N, K)
    pw = sq.prepare_weights_fp8b(w)
    wide = torch.full((M + 2, N + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[1:M + 1, 8:N + 8]
    assert sq.linear_fp8b(x, pw, out=out) is out
    xc, xs = ref.quant_rows(x)
    check_product(out, *ref.product(xc, xs, pw.W_8, pw.s_w))
    wide[1:M + 1, 8:N + 8] = 7.0
    assert bool((wide == 7.0).all()), "written outside of Y"
    sq.sq_check()


def test_linear_large_sampled():
    M, K, N = 4096, 4096, 6144
    x, w = activations(M, K), weights(N, K)
    layer = sq.SQBlockLinear(w)
    y = layer(x)
    xc, xs = ref.quant_rows(x)
    rows = torch.randperm(M, device=DEV, generator=gen(3))[:200]
    check_product(y[rows], *ref.product(xc[rows], xs[rows], layer.weights.W_8, layer.weights.s_w))
    assert torch.equal(layer(x), y)


def test_linear_blocks_of_zero_and_wide_scales():
    """Blocks that are all zero, and blocks whose scales differ by 2^60 (each must keep its own)."""
    M, K, N = 200, 640, 256
    x, w = activations(M, K).float(), weights(N, K).float()
    x[:, 128:256] = 0
    x[::2, 256:384] *= 2.0 ** 40
    x[:, 384:512] *= 2.0 ** -20
    w[128:, :128] = 0
    w[:128, 512:] *= 2.0 ** 20
    x, w = x.bfloat16(), w.bfloat16()
    for m in (M, 5):
        pw = sq.prepare_weights_fp8b(w)
        xc, xs = ref.quant_rows(x[:m])
        check_product(sq.linear_fp8b(x[:m], pw), *ref.product(xc, xs, pw.W_8, pw.s_w))


def test_linear_no_rows():
    pw = sq.prepare_weights_fp8b(weights(64, 136))
    assert sq.linear_fp8b(torch.empty(0, 136, dtype=torch.bfloat16, device=DEV), pw).shape == (0, 64)


# ------------------------------------------------------------------ routing
def check_route(logits, k, **kw):
    ids, w = sq.route(logits, k, **kw)
    rids, rw = ref.route(logits, k, **kw)
    assert torch.equal(ids.cpu(), rids)
    # fp32: exp of a rounded difference (its size in half steps), exp and division 4 half steps each, sums of up
    # to 512 + 16 terms in trees of at most 16 + 5 + 5 additions
    l = torch.nan_to_num(logits.float(), nan=-float("inf"), posinf=3.0e38, neginf=-float("inf"))
    spread = torch.where(l > -1e30, (l.amax(1, keepdim=True) - l).clamp(max=104.0), 0.0).max().item()
    tol = (2 * spread + 64) * 2.0 ** -24
    err = (w.double().cpu() - rw).abs()
    assert bool((err <= tol * rw + 1e-37 * kw.get("scale", 1.0)).all()), (err / rw.clamp_min(1e-37)).max()


ROUTES = [
    dict(k=1), dict(k=2, scoring="sigmoid"), dict(k=8, renormalize=False), dict(k=8, scoring="sigmoid", scale=2.5),
    dict(k=4, bias=True), dict(k=8, bias=True, scoring="sigmoid"),
    dict(k=4, groups=4, keep_groups=2), dict(k=4, groups=4, keep_groups=2, group_top=2),
    dict(k=8, groups=8, keep_groups=4, group_top=2, bias=True, scoring="sigmoid", scale=2.5),
    dict(k=3, groups=2, keep_groups=1, group_top=1, bias=True),
]


@pytest.mark.parametrize("kw", ROUTES)
@pytest.mark.parametrize("T,E", [(1, 16), (5, 40), (67, 64), (130, 256), (9, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(T, E, dtype, kw):
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = 0.1 * torch.randn(E, device=DEV, generator=gen(8))
    logits = (1.5 * torch.randn(T, E, device=DEV, generator=gen(T + E))).to(dtype)
    check_route(logits, **kw)


@pytest.mark.parametrize("kw", ROUTES)
def test_route_ties(kw):
    """Few distinct logits: every choice is among equals, and goes to the lower index."""
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = torch.arange(64, device=DEV).remainder(3).float() * 0.25
    logits = torch.randint(0, 3, (41, 64), device=DEV, generator=gen(2)).float()
    check_route(logits, **kw)
    check_route(torch.zeros_like(logits), **kw)


@pytest.mark.parametrize("kw", ROUTES)
def test_route_near_ties(kw):
    """Neighbouring fp32 logits, and saturated ones whose scores are equal in fp32 but not in fp64."""
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = torch.zeros(64, device=DEV)
    base = torch.randint(0, 4, (33, 64), device=DEV, generator=gen(4)).float() * 5.0 + 1.0
    step = torch.randint(-3, 4, (33, 64), device=DEV, generator=gen(5)).float() * 2.0 ** -23
    check_route(base * (1 + step), **kw)


@pytest.mark.parametrize("kw", ROUTES)
def test_route_masked(kw):
    """-inf, NaN and lowest logits; rows with fewer experts than choices, and with none."""
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = 0.1 * torch.randn(64, device=DEV, generator=gen(9))
    logits = torch.randn(40, 64, device=DEV, generator=gen(6))
    for t in range(40):
        dead = torch.randperm(64, device=DEV, generator=gen(100 + t))[: 64 - t // 2]
        logits[t, dead] = -float("inf") if t % 2 else float("nan")
    logits[30, 5] = torch.finfo(torch.float32).min
    logits[31, 7] = float("inf")
    check_route(logits, **kw)
    ids, w = sq.route(logits[:2], kw.pop("k"), **kw)
    assert bool((ids[:1] == -1).all()) and bool((w[:1] == 0).all())


def test_route_strided_logits():
    wide = torch.randn(50, 96, device=DEV, generator=gen(7))
    logits = wide[:, 16:80]
    ids, w = sq.route(logits, 6)
    ids2, w2 = sq.route(logits.contiguous(), 6)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    with pytest.raises(sq.SQError):
        sq.route(wide[:1].expand(50, 96), 6)


# ------------------------------------------------------------------ dispatch and combine
def some_ids(T, k, E, seed=0, holes=True):
    ids = torch.randint(0, E, (T, k), device=DEV, generator=gen(seed), dtype=torch.int32)
    if holes:
        r = torch.rand(T, k, device=DEV, generator=gen(seed + 1))
        ids = torch.where(r < 0.1, torch.full_like(ids, -1), ids)
        ids = torch.where(r > 0.97, torch.full_like(ids, E), ids)   # outside: no expert
    return ids


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 3, 7), (333, 4, 12), (1000, 8, 512), (4099, 8, 64), (31, 16, 300)])
def test_dispatch(T, k, E):
    for ids in (some_ids(T, k, E), torch.full((T, k), E - 1, dtype=torch.int32, device=DEV),
                torch.full((T, k), -1, dtype=torch.int32, device=DEV)):
        off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        pos = torch.empty(T, k, dtype=torch.int32, device=DEV)
        sq.sq_moe_dispatch(ids, E, off, pos)
        roff, rpos = ref.dispatch(ids, E)
        assert torch.equal(off.cpu(), roff) and torch.equal(pos.cpu(), rpos)


def test_moe_quant_scatters():
    T, k, E, K = 37, 3, 5, 264
    ids = some_ids(T, k, E)
    x = activations(T, K)
    gone = (ids < 0) | (ids >= E)
    x[gone.all(1)] = float("nan")    # a token without an expert is not read
    off, pos = (t.to(DEV) for t in ref.dispatch(ids, E))
    c = torch.full((T * k, 384), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((T * k, 4), 3.0, device=DEV)
    sq.sq_moe_quant_fp8b(x, pos, c, s)
    rc, rs = ref.quant_rows(x)
    ec, es = torch.full_like(c, 0x55), torch.full_like(s, 3.0)
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                ec[pos[t, j]], es[pos[t, j]] = rc[t], rs[t]
    assert torch.equal(c, ec) and torch.equal(s, es)


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (1, 8, 4096), (77, 3, 1032), (300, 16, 264)])
def test_combine(T, k, N):
    R = T * k
    pos = torch.randperm(R, device=DEV, generator=gen(1)).int().view(T, k)
    pos[torch.rand(T, k, device=DEV, generator=gen(2)) < 0.2] = -1
    z = torch.randn(R, N, device=DEV, generator=gen(3)).bfloat16()
    used = torch.zeros(R, dtype=torch.bool, device=DEV)
    used[pos[pos >= 0].long()] = True
    z[~used] = float("nan")           # rows of no choice are not read
    w = torch.rand(T, k, device=DEV, generator=gen(4))
    w[pos < 0] = float("nan")
    y = torch.full((T, N), 5.0, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_combine(z, pos, w, y)
    part = torch.where((pos >= 0).unsqueeze(-1), w.double().unsqueeze(-1) * z.double()[pos.clamp_min(0).long()], 0.0)
    total, mags = part.sum(1), part.abs().sum(1)
    lim = k * 2.0 ** -24 * mags + HALF_BF16 * (total.abs() + k * 2.0 ** -24 * mags)
    assert bool(((y.double() - total).abs() <= lim).all())


# ------------------------------------------------------------------ the experts' products
def rows_by_expert(counts):
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).int().to(DEV)
    return off, int(off[-1])


COUNTS = [[1], [0, 3, 0], [5, 0, 1, 16, 17, 0, 2], [130, 1, 0, 127], [40] * 9, [300, 12, 256, 0, 1], [700, 600],
          [300, 12, 700, 0, 1], [0, 0, 900, 0, 33], [1] * 33 + [0] * 40 + [64, 65]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", [(8, 8), (264, 136), (1024, 384), (512, 1160)])
def test_grouped_product(counts, K, N):
    off, rows = rows_by_expert(counts)
    E, R = len(counts), rows + 9        # rows behind the last expert's
    x = activations(R, K)
    pw = sq.prepare_weights_fp8b(weights(E, N, K))
    xc, xs = sq.quant_fp8b(x)
    y = torch.full((R, N + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_gemm_fp8b(xc, xs, off, pw.W_8, pw.s_w, N, K, y[:, :N])
    for e, n in enumerate(counts):
        a = int(off[e])
        if n:
            check_product(y[a:a + n, :N], *ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e], pw.s_w[e]))
    assert bool((y[rows:] == 7.0).all()) and bool((y[:, N:] == 7.0).all())
    sq.sq_check()


def check_swiglu(hc, hs, g, gm, u, um, I):
    """Codes and scales of h = silu(g) u against 64 bits: gm, um bound the products' magnitudes."""
    dg, du = ACC * gm, ACC * um
    sg = torch.sigmoid(g)
    h = g * sg * u
    # |d silu| <= 1.1; fp32 exp, sum, quotient and products: 16 half steps
    dh = 1.1 * dg * (u.abs() + du) + (g * sg).abs() * du + 16 * 2.0 ** -24 * h.abs()
    M = h.shape[0]
    kb = hs.shape[1]
    pad = ref.up(I, 128) - I
    hp = torch.nn.functional.pad(h, (0, pad)).view(M, -1, 128)
    dp = torch.nn.functional.pad(dh, (0, pad)).view(M, -1, 128)
    nb = hp.shape[1]
    amax = hp.abs().amax(2)
    da = dp.amax(2) + 2.0 ** -24 * amax
    s = hs[:, :nb].double()
    assert bool(((s - amax / 448).abs() <= da / 448 + 2.0 ** -23 * amax / 448).all()), "scales"
    assert bool((hs[:, nb:kb] == 0).all())
    v = ref.decode(hc).view(M, nb, 128)
    got = v * s.unsqueeze(2)
    # half an E4M3 step: 2^-4 of the value, 2^-10 of the scale for the smallest ones
    half = torch.maximum(2.0 ** -4 * hp.abs(), 2.0 ** -10 * s.unsqueeze(2))
    lim = half * (1 + 2.0 ** -10) + (1 + 2.0 ** -4) * dp + 2.0 ** -20 * hp.abs()
    assert bool(((got - hp).abs() <= lim).all()), "codes"
    assert bool((hc.view(M, -1)[:, I:] == 0).all()), "codes past I"


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,I", [(8, 8), (264, 136), (1024, 384), (512, 1160)])
def test_grouped_swiglu(counts, K, I):
    off, rows = rows_by_expert(counts)
    E, R = len(counts), rows + 5
    x = activations(R, K)
    pw = sq.prepare_weights_fp8b(weights(E, 2, I, K))
    xc, xs = sq.quant_fp8b(x)
    hc = torch.full((R, ref.up(I, 128)), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((R, ref.up(I, 512) // 128), 7.0, device=DEV)
    sq.sq_moe_swiglu_fp8b(xc, xs, off, pw.W_8, pw.s_w, I, K, hc, hs)
    for e, n in enumerate(counts):
        a = int(off[e])
        if n:
            g, gm = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 0], pw.s_w[e, 0])
            u, um = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 1], pw.s_w[e, 1])
            check_swiglu(hc[a:a + n], hs[a:a + n], g, gm, u, um, I)
    assert bool((hc[rows:] == 0x33).all()) and bool((hs[rows:] == 7.0).all())
    sq.sq_check()


# ------------------------------------------------------------------ the whole mixture
def staged(x, ids, w, gate_up, down):
    """experts_fp8b step by step through the public calls."""
    T, H = x.shape
    k, E, I = ids.shape[1], down.W_8.shape[0], gate_up.N
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    pos = torch.empty(T, k, dtype=torch.int32, device=DEV)
    sq.sq_moe_dispatch(ids, E, off, pos)
    xc = torch.empty(T * k, sq.sq_k_pad_fp8b(H), dtype=torch.uint8, device=DEV)
    xs = torch.empty(T * k, sq.sq_scale_ld_fp8b(H), device=DEV)
    sq.sq_moe_quant_fp8b(x, pos, xc, xs)
    hc = torch.empty(T * k, sq.sq_k_pad_fp8b(I), dtype=torch.uint8, device=DEV)
    hs = torch.empty(T * k, sq.sq_scale_ld_fp8b(I), device=DEV)
    sq.sq_moe_swiglu_fp8b(xc, xs, off, gate_up.W_8, gate_up.s_w, I, H, hc, hs)
    z = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_gemm_fp8b(hc, hs, off, down.W_8, down.s_w, H, I, z)
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_combine(z, pos, w, y)
    return y


def dense_mixture(x, ids, w, gate_up, down):
    """The mixture in 64 bits from the coded weights, h requantized as defined."""
    y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    xc, xs = ref.quant_rows(x)
    for e in range(down.W_8.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            g, _ = ref.product(xc[t], xs[t], gate_up.W_8[e, 0], gate_up.s_w[e, 0])
            u, _ = ref.product(xc[t], xs[t], gate_up.W_8[e, 1], gate_up.s_w[e, 1])
            hc, hs = ref.quant_rows(g * torch.sigmoid(g) * u)
            y.index_add_(0, t, ref.product(hc, hs, down.W_8[e], down.s_w[e])[0] * w[t, j].double().unsqueeze(1))
    return y


@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 256, 128), (16, 16, 300, 136, 128), (31, 8, 11, 520, 128), (32, 8, 9, 264, 136), (33, 8, 9, 264, 136),
                                       (1, 8, 64, 1024, 512), (9, 3, 7, 264, 136), (64, 4, 16, 512, 384),
                                       (333, 3, 12, 1032, 360), (700, 2, 4, 512, 640), (40, 1, 1, 128, 128)])
def test_experts(T, k, E, H, I):
    layer = sq.SQExperts(weights(E, 2 * I, H), weights(E, H, I, seed=2), k, scoring="sigmoid")
    x = activations(T, H)
    logits = torch.randn(T, E, device=DEV, generator=gen(5))
    if T > 5:
        logits[-3:] = -float("inf")      # a padded batch
        x[-3:] = float("nan")
    y = layer(x, logits)
    ids, w = sq.route(logits, k, scoring="sigmoid")
    assert torch.equal(y, staged(x, ids, w, layer.gate_up, layer.down))
    want = dense_mixture(x, ids, w, layer.gate_up, layer.down)
    # h's codes may differ by a step where its fp32 and 64-bit values fall on either side of a tie: 2^-3 of one of
    # I terms at the share of values within ACC of a tie; the experts' outputs are rounded to bf16 twice
    rel = ((y.double() - want).norm() / want.norm()).item()
    assert rel <= 2 * HALF_BF16, rel
    if T > 5:
        assert bool((y[-3:] == 0).all())
    sq.sq_check()


def test_experts_same_expert_twice():
    E, H, I = 3, 256, 128
    gu, dn = sq.prepare_weights_fp8b(weights(E, 2, I, H)), sq.prepare_weights_fp8b(weights(E, H, I, seed=2))
    x = activations(6, H)
    ids = torch.tensor([[0, 0], [1, 2], [2, 2], [0, 1], [1, 1], [-1, 2]], dtype=torch.int32, device=DEV)
    w = torch.rand(6, 2, device=DEV, generator=gen(1))
    y = sq.experts_fp8b(x, ids, w, gu, dn)
    want = dense_mixture(x, ids, w, gu, dn)
    assert ((y.double() - want).norm() / want.norm()).item() <= 2 * HALF_BF16


@pytest.mark.parametrize("T", [3, 300])
def test_captured_and_on_other_streams(T):
    """Two graphs and an eager call of the same layer, replayed at the same time on their own streams."""
    E, H, I, k = 8, 512, 256, 2
    layer = sq.SQExperts(weights(E, 2 * I, H), weights(E, H, I, seed=2), k)
    lin = sq.SQBlockLinear(weights(H, H, seed=3))
    xs = [activations(T, H, seed=s) for s in range(3)]
    ls = [torch.randn(T, E, device=DEV, generator=gen(s)) for s in range(3)]
    want = [lin(layer(x, l)) for x, l in zip(xs, ls)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, l in zip(xs[:2], ls[:2]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lin(layer(x, l)))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        y = layer(xs[2], ls[2], stream=side[2])
        y = lin(y, stream=side[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(y, want[2])
    sq.sq_check()


@pytest.mark.parametrize("M,K,N", [(1, 4096, 1048), (7, 1000, 264), (16, 8192, 520), (16, 136, 128), (3, 8, 8)])
def test_linear_is_its_two_steps(M, K, N):
    """Few rows are quantized inside the product: the same codes, scales and order of sums."""
    x, w = activations(M, K), weights(N, K)
    x[0, : min(128, K)] = 0
    x[-1, : min(8, K)] *= 2.0 ** -125
    pw = sq.prepare_weights_fp8b(w)
    xc, xs = sq.quant_fp8b(x)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    sq.sq_gemm_fp8b(xc, xs, pw.W_8, pw.s_w, M, N, K, y)
    assert torch.equal(sq.linear_fp8b(x, pw), y)
    wide = torch.zeros(M, K + 16, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:K + 8] = x
    assert torch.equal(sq.linear_fp8b(wide[:, 8:K + 8], pw), y)


def test_no_tokens_and_no_experts_left():
    E, H, I, k = 4, 136, 72, 2
    layer = sq.SQExperts(weights(E, 2, I, H), weights(E, H, I, seed=2), k)
    empty = torch.empty(0, H, dtype=torch.bfloat16, device=DEV)
    assert layer(empty, torch.empty(0, E, device=DEV)).shape == (0, H)
    x = activations(300, H)
    y = sq.experts_fp8b(x, torch.full((300, k), -1, dtype=torch.int32, device=DEV), torch.ones(300, k, device=DEV),
                        layer.gate_up, layer.down)
    assert bool((y == 0).all())
    sq.sq_check()


def test_prepared_round_trip():
    w = weights(200, 136)
    pw = sq.prepare_weights_fp8b(w)
    kept = {n: v.cpu() if torch.is_tensor(v) else v for n, v in pw.state_dict().items()}
    again = sq.PreparedFP8B.from_state_dict(kept, DEV)
    x = activations(20, 136)
    assert torch.equal(sq.linear_fp8b(x, again), sq.linear_fp8b(x, pw))


def test_weights_written_just_before():
    """Products fetch their first weights early: a preparation right before them in the stream still counts."""
    x = activations(4, 4096)
    a, b = weights(1024, 4096, seed=5), weights(1024, 4096, seed=6)
    pw = sq.prepare_weights_fp8b(a)
    want = [sq.linear_fp8b(x, sq.prepare_weights_fp8b(w)) for w in (a, b)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        sq.sq_prepare_weights_fp8b((a, b)[i % 2], pw.W_8, pw.s_w)
        got.append(sq.linear_fp8b(x, pw))
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


def test_refusals_on_the_gpu():
    pw = sq.prepare_weights_fp8b(weights(64, 136))
    x = activations(4, 136)
    with pytest.raises(ValueError):
        sq.linear_fp8b(x[:, :128], pw)                        # channels
    with pytest.raises(ValueError):
        sq.linear_fp8b(x, pw, out=torch.empty(4, 72, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        sq.linear_fp8b(x.float(), pw)
    with pytest.raises(sq.SQError) as e:                      # a row that does not start on 16 bytes
        sq.linear_fp8b(torch.zeros(4, 152, dtype=torch.bfloat16, device=DEV)[:, 4:140], pw)
    assert e.value.status == sq.SQ_ERR_MISALIGNED
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    gu, dn = sq.prepare_weights_fp8b(weights(2, 2, 64, 136)), sq.prepare_weights_fp8b(weights(2, 136, 64))
    with pytest.raises(TypeError):
        sq.experts_fp8b(x, ids, torch.ones(4, 2, device=DEV), gu, dn)
    with pytest.raises(ValueError):
        sq.experts_fp8b(x, ids.int(), torch.ones(4, 3, device=DEV), gu, dn)
    with pytest.raises(ValueError):
        sq.experts_fp8b(x, ids.int(), torch.ones(4, 2, device=DEV), dn, gu)


@pytest.mark.parametrize("M,K,N", [(64, 256, 16384), (65, 136, 16384), (100, 520, 16256), (100, 520, 16264),
                                   (128, 1032, 16392), (128, 128, 20480)])
def test_linear_where_the_kernel_changes(M, K, N):
    pw = sq.prepare_weights_fp8b(weights(N, K))
    x = activations(M, K)
    xc, xs = ref.quant_rows(x)
    check_product(sq.linear_fp8b(x, pw), *ref.product(xc, xs, pw.W_8, pw.s_w))


@pytest.mark.parametrize("rows", [64, 65, 100, 112, 113, 128, 130])
def test_grouped_product_where_the_kernel_changes(rows):
    """Experts of very different sizes around the mean that picks the kernel; rows behind the last one stay."""
    E, K, N, R = 33, 264, 520, 33 * rows
    cuts = torch.sort(torch.randint(0, R - 4, (E - 1,), generator=gen(rows), device=DEV)).values
    off = torch.cat([torch.zeros(1, device=DEV), cuts, torch.tensor([R - 5], device=DEV)]).int()
    pw = sq.prepare_weights_fp8b(weights(E, N, K))
    x = activations(R, K)
    xc, xs = sq.quant_fp8b(x)
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_gemm_fp8b(xc, xs, off, pw.W_8, pw.s_w, N, K, y)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            check_product(y[a:b], *ref.product(xc[a:b], xs[a:b], pw.W_8[e], pw.s_w[e]))
    assert bool((y[-5:] == 7.0).all())
    sq.sq_check()


def test_offsets_past_32_bits_linear():
    """More than 2^32 bytes of codes of x and of Y, more than 2^31 codes of W; the last rows and columns count."""
    M, K, N = 70016, 65536, 40064
    w = torch.randn(256, K, device=DEV, generator=gen(4)).bfloat16().repeat(N // 256 + 1, 1)[:N]
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 1, 32767, 32768, 65535, M - 130, M - 1], device=DEV)
    x[rows] = activations(len(rows), K)
    pw = sq.prepare_weights_fp8b(w)
    del w
    y = sq.linear_fp8b(x, pw)
    xc, xs = ref.quant_rows(x[rows])
    for lo in (0, (N // 2) // 128 * 128, N - 128):
        total, mags = ref.product(xc, xs, pw.W_8[lo:lo + 128], pw.s_w[lo // 128:lo // 128 + 1])
        check_product(y[rows, lo:lo + 128], total, mags)
    left = torch.ones(M, dtype=torch.bool, device=DEV)
    left[rows] = False
    assert not bool(y[left].any())
    sq.sq_check()
    del x, y, pw
    torch.cuda.empty_cache()


def test_offsets_past_32_bits_experts():
    """More than 2^32 codes of the pairs' rows; a token alone gives what it gives in the batch."""
    T, k, E, H, I = 66000, 16, 16, 4096, 128
    gu, dn = sq.prepare_weights_fp8b(weights(E, 2, I, H)), sq.prepare_weights_fp8b(weights(E, H, I, seed=2))
    x = activations(512, H).repeat(T // 512 + 1, 1)[:T]
    ids = torch.arange(16, dtype=torch.int32, device=DEV).repeat(T, 1)
    w = torch.rand(T, k, device=DEV, generator=gen(7))
    y = sq.experts_fp8b(x, ids, w, gu, dn)
    some = torch.tensor([0, 511, 32768, 65535, T - 1], device=DEV)
    want = dense_mixture(x[some], ids[some], w[some], gu, dn)
    rel = ((y[some].double() - want).norm(dim=1) / want.norm(dim=1)).max().item()
    assert rel <= 2 * HALF_BF16, rel
    sq.sq_check()
    del x, y, w, ids
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [3, 40, 64, 256, 512])
@pytest.mark.parametrize("kw", ROUTES)
def test_route_zeros_of_both_signs(E, kw, dtype):
    """-0.0 and +0.0 are the same logit: a tie inside a group and between groups (whose best scores they may be)."""
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = torch.zeros(E, device=DEV).copysign(torch.randn(E, device=DEV, generator=gen(3)))
    if kw["k"] > E // kw.get("groups", 1) * kw.get("keep_groups", 1) or E % kw.get("groups", 1):
        kw = dict(k=1)
    pick = torch.randint(0, 3, (37, E), device=DEV, generator=gen(E))
    logits = torch.tensor([0.0, -0.0, -1.0], device=DEV)[pick].to(dtype)
    logits[0, :3] = torch.tensor([-0.0, 0.0, -1.0], device=DEV)
    check_route(logits, **kw)
    check_route(-torch.zeros_like(logits), **kw)


def check_route_order(logits, k, bias, groups, keep_groups, scoring="softmax"):
    """ids against 64 bits for many tokens (group_top 2); the scores are too varied to tie."""
    T, E = logits.shape
    l = logits.double()
    score = (torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)) + bias.double()
    by_group = score.view(T, groups, E // groups)
    kept = by_group.topk(2, 2).values.sum(2).topk(keep_groups, 1).indices
    open_ = torch.zeros(T, groups, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
    score = by_group.masked_fill(~open_.unsqueeze(2), -float("inf")).flatten(1)
    ids, _ = sq.route(logits, k, bias=bias, scoring=scoring, groups=groups, keep_groups=keep_groups, group_top=2)
    assert torch.equal(ids.long(), score.topk(k, 1).indices)


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (512, 4), (40, 4), (96, 16)])   # groups of whole lanes, and others
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [256.0, 1000.0, 4096.0])
def test_route_groups_whose_scores_cancel(E, groups, scoring, big):
    """A group's two best scores are about +B and -B: its sum is small, the error of their fp32 values is not."""
    per, T = E // groups, 16384
    bias = torch.full((groups, per), -16 * big, device=DEV)
    for g in range(groups):
        a, c = torch.randperm(per, device=DEV, generator=gen(g))[:2].tolist()
        bias[g, a], bias[g, c] = big, -big
    if groups == 8:
        bias[3, bias[3].abs() <= big] = 0.0      # a group whose scores are small among those that are not
    logits = 1.5 * torch.randn(T, E, device=DEV, generator=gen(E))
    for keep in (1, groups // 2):
        check_route_order(logits, min(4, 2 * keep), bias.flatten().contiguous(), groups, keep, scoring)


@pytest.mark.parametrize("counts", [[16], [9] * 40, [60] * 5, [300], [129, 0, 520]])
@pytest.mark.parametrize("I", [136, 1160])
def test_swiglu_of_tiny_rows(counts, I):
    """Rows whose h ends near and below the smallest fp32 number: a scale that rounds to 0 has zero codes, nothing is
    NaN, and the rows beside them keep their values."""
    off, R = rows_by_expert(counts)
    E, K = len(counts), 264
    power = torch.arange(R, device=DEV) % 12
    x = torch.randn(R, K, device=DEV, generator=gen(1)) * torch.where(power > 0, 2.0 ** -(65.0 + power), 1.0).unsqueeze(1)
    pw = sq.prepare_weights_fp8b(weights(E, 2, I, K))
    xc, xs = sq.quant_fp8b(x.bfloat16())
    hc = torch.full((R, ref.up(I, 128)), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((R, ref.up(I, 512) // 128), 7.0, device=DEV)
    sq.sq_moe_swiglu_fp8b(xc, xs, off, pw.W_8, pw.s_w, I, K, hc, hs)
    sq.sq_check()
    got = ref.rows64(hc, hs)[:, :I]
    for e, n in enumerate(counts):
        if n == 0:
            continue
        a = int(off[e])
        g, gm = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 0], pw.s_w[e, 0])
        u, um = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 1], pw.s_w[e, 1])
        sg = torch.sigmoid(g)
        h = g * sg * u
        dh = 1.1 * ACC * gm * (u.abs() + ACC * um) + (g * sg).abs() * ACC * um + 2.0 ** -18 * h.abs()
        dh += 2.0 ** -149 * (1 + u.abs())     # silu and h are rounded to fp32's steps
        top = torch.nn.functional.pad(h.abs() + dh, (0, -I % 128)).view(n, -1, 128).amax(2).repeat_interleave(128, 1)[:, :I]
        # half an E4M3 step of the value, 2^-10 of the scale at least; the scale is off by half an fp32 step, 2^-150 at
        # least, at up to 448 times that; values up to the block's largest one
        lim = torch.maximum(2.0 ** -4 * (h.abs() + dh), 2.0 ** -10 * top / 448) + dh + 2.0 ** -23 * top + 2 * 448 * 2.0 ** -150
        err = (got[a:a + n] - h).abs()
        assert bool((err <= lim).all()), "h"      # (false for NaN)
    none = hs == 0
    codes = hc.view(R, -1, 128)
    assert bool((codes[none[:, :codes.shape[1]]] == 0).all()), "codes of a zero scale"
    assert bool(none[:, 0].any()) and not bool(none[:, 0].all())


@pytest.mark.parametrize("T", [2, 40, 700])
def test_experts_of_tiny_tokens(T):
    E, H, I, k = 4, 264, 136, 2
    layer = sq.SQExperts(weights(E, 2, I, H), weights(E, H, I, seed=2), k)
    x = activations(T, H)
    logits = torch.randn(T, E, device=DEV, generator=gen(5))
    want = layer(x, logits)
    small = x.clone()
    small[::2] *= 2.0 ** -74
    y = layer(small, logits)
    assert bool((y[::2].abs() <= 1e-38).all())      # (false for NaN)
    assert torch.equal(y[1::2], want[1::2])


def test_prepare_weights_stack_of_strided_matrices():
    """Leading dimensions that no single stride runs through."""
    E, I, K = 3, 200, 264
    wide = weights(E, 2 * I + 24, K + 16)
    w = wide[:, 8:2 * I + 8, 8:K + 8]
    stack = w.reshape(E, 2, I, K)
    assert stack.data_ptr() == w.data_ptr()           # a view, not a copy
    pw, want = sq.prepare_weights_fp8b(stack), sq.prepare_weights_fp8b(stack.contiguous())
    assert torch.equal(pw.W_8, want.W_8) and torch.equal(pw.s_w, want.s_w)
    turned = weights(2, E, I, K).transpose(0, 1)
    pw, want = sq.prepare_weights_fp8b(turned), sq.prepare_weights_fp8b(turned.contiguous())
    assert torch.equal(pw.W_8, want.W_8) and torch.equal(pw.s_w, want.s_w)
    down = weights(E, K, I, seed=2)
    layer, same = sq.SQExperts(w, down, 2), sq.SQExperts(w.contiguous(), down, 2)
    x, logits = activations(5, K), torch.randn(5, E, device=DEV, generator=gen(5))
    assert torch.equal(layer(x, logits), same(x, logits))


@pytest.mark.parametrize("E", [164, 165, 256, 384, 459, 460, 512])
@pytest.mark.parametrize("mean", [2, 9, 24])
def test_grouped_products_of_many_experts(E, mean):
    """Where the experts' tables leave room for one CTA on an SM and not for two."""
    K, I = 136, 264
    counts = torch.randint(0, 2 * mean + 1, (E,), generator=gen(E), device=DEV).tolist()
    off, R = rows_by_expert(counts)
    x = activations(R, K)
    xc, xs = sq.quant_fp8b(x)
    pw = sq.prepare_weights_fp8b(weights(E, 2, I, K))
    y = torch.empty(R, I, dtype=torch.bfloat16, device=DEV)
    sq.sq_moe_gemm_fp8b(xc, xs, off, pw.W_8[:, 0].contiguous(), pw.s_w[:, 0].contiguous(), I, K, y)
    hc = torch.full((R, ref.up(I, 128)), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((R, ref.up(I, 512) // 128), 7.0, device=DEV)
    sq.sq_moe_swiglu_fp8b(xc, xs, off, pw.W_8, pw.s_w, I, K, hc, hs)
    sq.sq_check()
    for e, n in enumerate(counts):
        if n:
            a = int(off[e])
            g, gm = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 0], pw.s_w[e, 0])
            u, um = ref.product(xc[a:a + n], xs[a:a + n], pw.W_8[e, 1], pw.s_w[e, 1])
            check_product(y[a:a + n], g, gm)
            check_swiglu(hc[a:a + n], hs[a:a + n], g, gm, u, um, I)


@pytest.mark.parametrize("M,K,N", [
    (1, 8192, 8192), (16, 136, 128), (3, 8, 8),             # K split over clusters; one block; fewer than the ring holds
    (16, 264, 40960), (30, 1032, 40960), (5, 128, 57344),   # persistent: several tiles a CTA, one block to nine
    (33, 4096, 1048), (64, 264, 16384), (100, 4104, 520), (128, 384, 8192)])   # tiles of 64 and of 128 rows
def test_early_weights_change_nothing(M, K, N):
    """The product behind the quantizer fetches its first weights before its wait; called alone it waits first."""
    x = activations(M, K)
    pw = sq.prepare_weights_fp8b(weights(N, K))
    xc, xs = sq.quant_fp8b(x)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    sq.sq_gemm_fp8b(xc, xs, pw.W_8, pw.s_w, M, N, K, y)
    for _ in range(3):
        assert torch.equal(sq.linear_fp8b(x, pw), y)


def test_offsets_past_32_bits_of_distinct_weights():
    """Blocks at the start, in the middle and at the end of more than 2^31 codes of W, none like another: each is
    prepared as by itself and gives its own columns of more than 2^32 bytes of Y, in the products for many rows and for few."""
    M, K, N = 60032, 65536, 40064
    at = (0, 16384, 32768, N // 2 // 128 * 128, N - 128)
    w = torch.randn(256, K, device=DEV, generator=gen(4)).bfloat16().repeat(N // 256 + 1, 1)[:N]
    for i, lo in enumerate(at):
        w[lo:lo + 128] = weights(128, K, seed=20 + i) * 2.0 ** i
    pw = sq.prepare_weights_fp8b(w)
    for lo in at:
        wc, ws = ref.quant_weights(w[lo:lo + 128])
        assert torch.equal(pw.W_8[lo:lo + 128], wc) and torch.equal(pw.s_w[lo // 128], ws[0])
    del w
    rows = torch.tensor([0, 1, 32768, 53000, M - 130, M - 1], device=DEV)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[rows] = activations(len(rows), K)
    xc, xs = ref.quant_rows(x[rows])
    many, few = sq.linear_fp8b(x, pw)[rows], sq.linear_fp8b(x[rows], pw)
    for lo in at:
        total, mags = ref.product(xc, xs, pw.W_8[lo:lo + 128], pw.s_w[lo // 128:lo // 128 + 1])
        check_product(many[:, lo:lo + 128], total, mags)
        check_product(few[:, lo:lo + 128], total, mags)
    sq.sq_check()
    del x, pw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,K", [(200, 520), (128, 512), (264, 136)])
def test_weights_quantized_elsewhere(N, K):
    """Codes [N, K] and scales [ceil(N / 128), ceil(K / 128)] padded to the library's shapes."""
    pw = sq.prepare_weights_fp8b(weights(N, K))
    codes = pw.W_8[:, :K].contiguous().view(torch.float8_e4m3fn)
    scales = pw.s_w[:, :-(-K // 128)].contiguous()
    pad = torch.nn.functional.pad
    again = sq.PreparedFP8B(N, K, pad(codes.view(torch.uint8), (0, sq.sq_k_pad_fp8b(K) - K)),
                            pad(scales, (0, sq.sq_scale_ld_fp8b(K) - scales.shape[-1])))
    x = activations(20, K)
    assert torch.equal(sq.linear_fp8b(x, again), sq.linear_fp8b(x, pw))


@pytest.mark.parametrize("kw", [dict(k=4), dict(k=8, scoring="sigmoid"), dict(k=4, groups=4, keep_groups=2),
                                dict(k=6, groups=8, keep_groups=4, group_top=2, scoring="sigmoid")])
def test_route_bias_of_minus_infinity(kw):
    """Experts of bias -inf come after all others, in the order of their index; a group's worth may be -inf."""
    bias = 0.1 * torch.randn(64, device=DEV, generator=gen(9))
    bias[torch.randperm(64, device=DEV, generator=gen(10))[:50]] = -float("inf")
    bias[:16] = -float("inf")
    check_route(1.5 * torch.randn(40, 64, device=DEV, generator=gen(11)), bias=bias, **kw)
    check_route(1.5 * torch.randn(4, 64, device=DEV, generator=gen(12)), bias=torch.full_like(bias, -float("inf")), **kw)
