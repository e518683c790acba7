"""Block-FP8 products with an epilogue: the dense product with bias, activation
and residual, its gradient, the experts' grouped products, and a whole expert
layer, against definitions in 64 bits.

Tolerance of a product before its epilogue, from the kernels' arithmetic: the
products of E4M3 values are exact, a k-block's 128 are summed in f32 by the
tensor core (at most a rounding per addition, 128 * 2^-23 of the sum of sizes),
its scale is one rounding and it enters the f32 sum by one fused multiply-add:
with T = sum_b |sa sw| sum_k |a w| that is T (2^-16 + (nkb + 1) 2^-24), and the
bias adds a rounding of the sum. Through the activation an error d before it is
at most 1.13 d after it (the largest slope of the gelus and silu), and the
activation itself adds 2^-19 (|z| + |act(z)|): an exponential and a reciprocal
of 2 ulp each, a relative error of the exponential that grows by |x| 2^-23
where the function falls as exp(-|x|), or erf's 2 ulp beside 1. Half a step of
the result's type is eps / 2 relative."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def bq():
    import dequantize_absmax_reduce_b200 as m
    assert torch.cuda.is_available()
    return m


def half_step(t, dtype):
    fi = torch.finfo(dtype)
    return t.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def after_act(z, d, act):
    """act(z) and the error it may carry, for a z that is off by at most d."""
    v = act64(z, act)
    if act in ("none", "relu"):
        return v, d
    return v, 1.13 * d + 2.0 ** -19 * (z.abs() + v.abs())


def codes(shape, g, rows):
    """Random E4M3 codes (all finite ones) and scales of blocks of `rows` x 128."""
    c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
    c[(c & 127) == 127] = 0x38
    s = torch.rand((*shape[:-2], -(-shape[-2] // rows), shape[-1] // 128), generator=g) * 0.002 + 0.0005
    return c.cuda(), s.cuda()


def values(c, s, rows):
    s = s.double().repeat_interleave(128, -1)
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., :c.shape[-2], :]
    return c.view(F8).double() * s


def product(a, w, nkb):
    """(A W^T, its error bound) in 64 bits."""
    t = a.abs() @ w.abs().t()
    return a @ w.t(), t * (2.0 ** -16 + (nkb + 1) * 2.0 ** -24) * (1 + 2.0 ** -20)


def bound_check(got, ref, err, dtype, what):
    assert got.dtype == dtype
    bad = (got.double() - ref).abs() > err * (1 + 2.0 ** -18) + half_step(ref.abs() + err, dtype)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


# ---------------------------------------------------------------- dense
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (1, 129, 256), (7, 1000, 384), (16, 4096, 2048), (33, 65, 128), (128, 256, 128), (129, 257, 512),
                                   (300, 520, 512), (257, 384, 1024), (1000, 2050, 256)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [BF, HF, F32])
def test_epilogue(bq, m, n, k, act, out):
    g = torch.Generator().manual_seed(m + n + k)
    a, sa = codes((m, k), g, 1)
    w, sw = codes((n, k), g, 128)
    z, d = product(values(a, sa, 1), values(w, sw, 128), k // 128)
    std = z.std().item() + 1e-3
    for with_bias, with_res, with_pre in ((BF, True, True), (F32, False, False), (None, True, False), (HF, False, True)):
        bias = None if with_bias is None else (std * torch.randn(n, generator=g)).to(with_bias).cuda()
        res = (std * torch.randn((m, n), generator=g)).to(out).cuda() if with_res else None
        got = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, act, res, out, with_pre)
        zb = z if bias is None else z + bias.double()
        db = d + 2.0 ** -24 * (zb.abs() + d)
        v, dv = after_act(zb, db, act)
        if with_pre:
            got, pre = got
            bound_check(pre, zb, db, out, "pre")
        if with_res:
            v = v + res.double()
            dv = dv + 2.0 ** -24 * (v.abs() + dv)
        bound_check(got, v, dv, out, f"{m}x{n}x{k} {act} {with_bias} {with_res}")


def test_epilogue_without_extras_is_the_product(bq):
    """No bias, no activation, no residual: the bits of bq_fp8_block_gemm_quantized, where one CTA sums all of k (products of
    few tiles and at least four k-blocks are shared by CTAs, whose sums are joined in another order: test_epilogue has those)."""
    g = torch.Generator().manual_seed(4)
    for m, n, k in ((5, 300, 384), (128, 512, 256), (1300, 1100, 640), (2000, 3000, 640)):
        a, sa = codes((m, k), g, 1)
        w, sw = codes((n, k), g, 128)
        for out in (BF, F32):
            assert torch.equal(bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, out_dtype=out),
                               bq.api.fp8_block_gemm_quantized(a, sa, w, sw, out))


def test_epilogue_residual_in_place_and_repeated(bq):
    g = torch.Generator().manual_seed(6)
    a, sa = codes((300, 512), g, 1)
    w, sw = codes((700, 512), g, 128)
    res = torch.randn((300, 700), generator=g).bfloat16().cuda()
    want = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, None, "silu", res)
    for _ in range(3):
        assert torch.equal(bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, None, "silu", res), want)
    bq._bq.bq_fp8_block_gemm_epilogue(a, sa, w, sw, res, None, "silu", res)
    assert torch.equal(res, want)


def test_epilogue_special_values(bq):
    """Large and infinite arguments of the activations, NaN codes, zero scales: as the formulas say."""
    g = torch.Generator().manual_seed(8)
    a, sa = codes((40, 256), g, 1)
    w, sw = codes((96, 256), g, 128)
    a[3, 7] = 0x7F                                # NaN: its row
    sa[5] = 0.0                                   # a row of zeros
    bias = torch.zeros(96)
    bias[0], bias[1], bias[2], bias[3] = 1e30, -1e30, math.inf, 3e38
    for act in ACTS:
        c = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias.cuda(), act, out_dtype=F32)
        assert torch.isnan(c[3]).all() and not torch.isnan(torch.cat([c[:3], c[4:]])).any()
        ok = torch.cat([c[:3], c[4:]])
        assert (ok[:, 0] == torch.tensor(1e30)).all() and (ok[:, 2] == math.inf).all() and (ok[:, 3] == torch.tensor(3e38)).all()
        assert (ok[:, 1] == (torch.tensor(-1e30) if act == "none" else 0)).all()
        assert (c[5, 4:] == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (3, 100), (31, 256), (33, 7), (200, 2056), (1025, 264), (4097, 40)])
def test_epilogue_backward(bq, act, dtype, m, n):
    g = torch.Generator().manual_seed(m * n)
    dy = torch.randn((m, n), generator=g).to(dtype).cuda()
    pre = (2.0 * torch.randn((m, n), generator=g)).to(dtype).cuda()
    if m > 2 and n > 2:
        pre[0, 0], pre[1, 1], pre[2, 2], pre[0, 1] = 0.0, 60000.0, -60000.0, -30.0
    z = pre.double().requires_grad_(True)
    act64(z, act).backward(dy.double()) if act != "relu" else (torch.where(z > 0, z, 0.0)).backward(dy.double())
    ref = z.grad
    dz, db = bq.api.gemm_epilogue_backward(dy, pre, act)
    # The slope is at most 1.13 in size; its terms carry at most 2^-19 of 1 + |z| while z^2 < 64, beyond which s (1 - s) z has vanished.
    err = 2.0 ** -19 * dy.double().abs() * (1 + pre.double().abs().clamp_max(8.0))
    if act in ("none", "relu"):
        err = torch.zeros_like(err)
    bound_check(dz, ref, err, dtype, "dz")
    size = ref.abs() + err
    assert ((db.double() - ref.sum(0)).abs() <= err.sum(0) + m * 2.0 ** -24 * size.sum(0) + 1e-300).all()
    dz2, none = bq.api.gemm_epilogue_backward(dy, pre, act, bias_grad=False)
    assert none is None and torch.equal(dz2, dz)
    again = bq.api.gemm_epilogue_backward(dy, pre, act)
    assert torch.equal(again[1], db)
    bq._bq.bq_gemm_epilogue_backward(dy, pre, act, dy)            # in place
    assert torch.equal(dy, dz)


def test_epilogue_backward_against_differences(bq):
    """The slope against central differences of the forward kernel: one code row and a bias sweep give act at known points."""
    a = torch.zeros((1, 128), dtype=torch.uint8, device="cuda")
    sa = torch.ones((1, 1), device="cuda")
    w = torch.zeros((512, 128), dtype=torch.uint8, device="cuda")
    sw = torch.ones((4, 1), device="cuda")
    z = torch.linspace(-6, 6, 512)
    z = (z * 1024).round() / 1024
    h = 2.0 ** -6
    for act in ACTS:
        f = lambda b: bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, b.cuda(), act, out_dtype=F32).double().cpu()[0]   # noqa: E731
        slope = (f(z + h) - f(z - h)) / (2 * h)
        dz, db = bq.api.gemm_epilogue_backward(torch.ones((1, 512), device="cuda"), z.cuda()[None], act)
        assert torch.equal(dz[0], db)
        # Third derivatives are below 3; values to 2^-18 of 1 + |z|; relu has its corner within h of 0.
        bound = h * h / 6 * 3 + 2.0 ** -18 * (1 + z.double().abs()) / h
        away = (z.abs() > h) if act == "relu" else torch.ones_like(z, dtype=torch.bool)
        assert ((slope - dz[0].double().cpu()).abs() <= bound)[away].all(), act


# ---------------------------------------------------------------- experts
def grouped_ref(a, sa, rows, off, w, sw, bias, act, gated):
    va, nkb = values(a, sa, 1), a.shape[1] // 128
    parts = []
    for e in range(len(off) - 1):
        here = slice(off[e], off[e + 1])
        x = va[here] if rows is None else va[rows[here].long()]
        z, d = product(x, values(w[e], sw[e], 128), nkb)
        if bias is not None:
            z = z + bias[e].double()
        d = d + 2.0 ** -24 * (z.abs() + d)
        if gated:
            h = z.shape[1] // 2
            v, dv = after_act(z[:, :h], d[:, :h], act)
            u, du = z[:, h:], d[:, h:]
            z, d = v * u, dv * u.abs() + v.abs() * du + dv * du
            d = d + 2.0 ** -24 * (z.abs() + d)
        else:
            z, d = after_act(z, d, act)
        parts.append((z, d))
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def offsets_of(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("counts,n,k", [([1], 256, 128), ([0, 3, 0, 0, 1, 0], 256, 256), ([5, 0, 130, 128, 127, 1], 512, 384),
                                        ([0, 0, 0], 256, 128), ([2] * 40, 256, 512), ([300, 17, 0, 260], 768, 1024), ([1, 2, 3, 4, 33, 64, 96, 31], 1280, 640)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(bq, counts, n, k, gated, gather):
    g = torch.Generator().manual_seed(sum(counts) + n + k)
    e = len(counts)
    off, offsets = offsets_of(counts)
    p = off[-1]
    behind = 3
    t = max(1, p // 2) if gather else p + behind
    a, sa = codes((t, k), g, 1)
    w, sw = codes((e, n, k), g, 128)
    rows = torch.randint(0, t, (p + behind,), generator=g).to(torch.int32).cuda() if gather else None
    for act, with_bias, out in (("silu", False, BF), ("none", True, F32), ("gelu", True, HF), ("gelu_tanh", False, F32), ("relu", True, BF)):
        bias = torch.randn((e, n), generator=g).to(BF if act == "relu" else F32).cuda() if with_bias else None
        c = torch.full((p + behind, n // 2 if gated else n), 9.0, dtype=out, device="cuda")
        got = bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, rows, bias, act, gated, out=c)
        assert got is c and (c[p:] == 9.0).all()                  # rows behind the last expert's stay
        if p:
            ref, err = grouped_ref(a, sa, rows, off, w, sw, bias, act, gated)
            # A gated product of two large factors can pass f16's range: rounding to infinity is the type's.
            keep = ref.abs() < (60000 if out == HF else 1e38)
            bound_check(torch.where(keep, c[:p], 0.0), torch.where(keep, ref, 0.0), torch.where(keep, err, 0.0), out, f"{act} {gated}")


@pytest.mark.parametrize("n", [1, 3, 63, 64, 127, 128, 130, 1000])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_grouped_odd_widths(bq, n, act):
    """Columns that end inside a tile: the next expert's weights follow in memory."""
    g = torch.Generator().manual_seed(n)
    counts = [3, 0, 40, 129]
    off, offsets = offsets_of(counts)
    a, sa = codes((off[-1], 256), g, 1)
    w, sw = codes((4, n, 256), g, 128)
    bias = torch.randn((4, n), generator=g).cuda()
    for out in (BF, F32):
        c = bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, None, bias, act, out_dtype=out)
        bound_check(c, *grouped_ref(a, sa, None, off, w, sw, bias, act, False), out, f"n {n}")


def test_grouped_many_experts(bq):
    """More experts than the kernel's table has entries, most of them without a row."""
    g = torch.Generator().manual_seed(12)
    for e in (256, 257, 700, 1024):
        counts = (torch.rand(e, generator=g) < 0.3).long() * torch.randint(1, 5, (e,), generator=g)
        counts[-1] = 2
        off, offsets = offsets_of(counts.tolist())
        a, sa = codes((off[-1], 128), g, 1)
        w, sw = codes((e, 64, 128), g, 128)
        c = bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, out_dtype=F32)
        bound_check(c, *grouped_ref(a, sa, None, off, w, sw, None, "none", False), F32, f"{e} experts")


def test_grouped_bad_indexes_stay_inside(bq):
    """Activation rows outside the tensor count as zeros; offsets past the positions or falling are bounded."""
    g = torch.Generator().manual_seed(13)
    a, sa = codes((20, 256), g, 1)
    w, sw = codes((3, 256, 256), g, 128)
    rows = torch.arange(20, dtype=torch.int32)
    rows[4], rows[9], rows[15] = -7, 20, 2 ** 31 - 1
    off = torch.tensor([0, 8, 8, 20], dtype=torch.int32, device="cuda")
    c = bq.api.fp8_grouped_gemm(a, sa, off, w, sw, rows.cuda(), out_dtype=F32)
    good = bq.api.fp8_grouped_gemm(a, sa, off, w, sw, torch.arange(20, dtype=torch.int32, device="cuda"), out_dtype=F32)
    bad = torch.tensor([4, 9, 15])
    keep = torch.ones(20, dtype=torch.bool)
    keep[bad] = False
    assert (c[bad.cuda()] == 0).all() and torch.equal(c[keep.cuda()], good[keep.cuda()])
    out = torch.full((20, 256), 5.0, device="cuda")
    bq.api.fp8_grouped_gemm(a, sa, torch.tensor([-3, 8, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), w, sw, out=out)
    assert torch.equal(out[:5], good[:5])          # [0, 8) of the first, none of the second, [5, 20) of the third
    ref = bq.api.fp8_grouped_gemm(a, sa, torch.tensor([0, 0, 0, 20], dtype=torch.int32, device="cuda"), w, sw, out_dtype=F32)
    assert torch.equal(out[8:], ref[8:])


def test_grouped_one_expert_is_the_dense_product(bq):
    g = torch.Generator().manual_seed(14)
    a, sa = codes((333, 640), g, 1)
    w, sw = codes((1, 520, 640), g, 128)
    off = torch.tensor([0, 333], dtype=torch.int32, device="cuda")
    assert torch.equal(bq.api.fp8_grouped_gemm(a, sa, off, w, sw), bq.api.fp8_block_gemm_quantized(a, sa, w[0], sw[0]))


def test_grouped_many_tiles(bq):
    """Several tiles per CTA through the same rings, in a shape of long runs."""
    g = torch.Generator().manual_seed(15)
    counts = [700, 0, 1300, 41, 512, 2000, 129, 256]
    off, offsets = offsets_of(counts)
    a, sa = codes((900, 512), g, 1)
    w, sw = codes((8, 2048, 512), g, 128)
    rows = torch.randint(0, 900, (off[-1],), generator=g).to(torch.int32).cuda()
    c = bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, rows, act="silu", gated=True)
    ref, err = grouped_ref(a, sa, rows, off, w, sw, None, "silu", True)
    bound_check(c, ref, err, BF, "many tiles")


# ---------------------------------------------------------------- a whole layer
def layer_ref(bq, x, logits, w1, s1, w2, s2, top_k, **kw):
    ids, wt = bq.api.moe_route(logits, top_k, **{k: v for k, v in kw.items() if k in ("bias", "score", "n_groups", "top_groups", "scale")})
    ea, sa = bq.api.fp8_block_quantize(x, 1, 128)
    va = values(ea, sa, 1)
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    first = kw.get("first_expert", 0)
    for e in range(w1.shape[0]):
        t, j = (ids == e + first).nonzero(as_tuple=True)
        if not t.numel():
            continue
        z = va[t] @ values(w1[e], s1[e], 128).t()
        h = act64(z[:, :z.shape[1] // 2], "silu") * z[:, z.shape[1] // 2:]
        out.index_add_(0, t, wt[t, j].double()[:, None] * (h @ values(w2[e], s2[e], 128).t()))
    return out


@pytest.mark.parametrize("t", [1, 5, 300])
def test_layer(bq, t):
    """Routing, order, products, quantization between them and the sum, against the layer in 64 bits without the middle
    quantization: that is a relative error of at most 2^-4 per value of h, and sums of many such errors of either sign;
    with h and the weights' values independent their size is about 2^-4 / sqrt(3) of the result's, here bounded by 2^-4."""
    g = torch.Generator().manual_seed(t)
    h, inter, e, k = 512, 256, 16, 4
    x = torch.randn((t, h), generator=g).bfloat16().cuda()
    logits = torch.randn((t, e), generator=g).cuda()
    bias = (0.1 * torch.randn(e, generator=g)).cuda()
    w1, s1 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * 2 * inter, h), generator=g)).bfloat16().cuda(), 128)
    w2, s2 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * h, inter), generator=g)).bfloat16().cuda(), 128)
    w1, s1 = w1.view(e, 2 * inter, h), s1.view(e, 2 * inter // 128, h // 128)
    w2, s2 = w2.view(e, h, inter), s2.view(e, h // 128, inter // 128)
    kw = {"bias": bias, "score": "sigmoid", "n_groups": 4, "top_groups": 2, "scale": 2.5}
    res = torch.randn((t, h), generator=g).bfloat16().cuda()
    full = bq.api.fp8_moe(x, logits, w1, s1, w2, s2, k, **kw)
    ref = layer_ref(bq, x, logits, w1, s1, w2, s2, k, **kw)
    assert (full.double() - ref).norm() <= 2.0 ** -4 * ref.norm()
    with_res = bq.api.fp8_moe(x, logits, w1, s1, w2, s2, k, residual=res, **kw)
    assert ((with_res.double() - res.double() - full.double()).abs() <= half_step(with_res.double(), BF) + half_step(full.double(), BF) + 1e-6).all()
    # The experts' halves on two GPUs add up to the layer.
    halves = [bq.api.fp8_moe(x, logits, w1[a:b], s1[a:b], w2[a:b], s2[a:b], k, first_expert=a, **kw) for a, b in ((0, 8), (8, 16))]
    parts = [layer_ref(bq, x, logits, w1[a:b], s1[a:b], w2[a:b], s2[a:b], k, first_expert=a, **kw) for a, b in ((0, 8), (8, 16))]
    for got, want in zip(halves, parts):
        assert (got.double() - want).norm() <= 2.0 ** -4 * want.norm() + 1e-30
    assert ((halves[0].double() + halves[1].double() - full.double()).abs()
            <= half_step(halves[0].double(), BF) + half_step(halves[1].double(), BF) + half_step(full.double(), BF) + 1e-5).all()


def test_layer_with_masked_tokens(bq):
    """Padded tokens (every logit -inf) come out as their residual alone, whatever their activations hold."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn((6, 256), generator=g).bfloat16().cuda()
    logits = torch.randn((6, 8), generator=g).cuda()
    logits[2] = logits[5] = -math.inf
    x[2] = math.nan
    w1, s1 = codes((8, 512, 256), g, 128)
    w2, s2 = codes((8, 256, 256), g, 128)
    res = torch.randn((6, 256), generator=g).bfloat16().cuda()
    out = bq.api.fp8_moe(x, logits, w1, s1, w2, s2, 2, residual=res)
    assert torch.equal(out[[2, 5]], res[[2, 5]]) and torch.isfinite(out).all()


def test_layer_in_a_graph_and_on_streams(bq):
    """Captured once, replayed on new inputs; and on two streams at once."""
    g = torch.Generator().manual_seed(3)
    h, e, k = 256, 8, 2
    w1, s1 = codes((e, 512, h), g, 128)
    w2, s2 = codes((e, h, 256), g, 128)
    x = torch.randn((70, h), generator=g).bfloat16().cuda()
    logits = torch.randn((70, e), generator=g).cuda()
    run = lambda x, l: bq.api.fp8_moe(x, l, w1, s1, w2, s2, k, score="sigmoid")   # noqa: E731
    run(x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x, logits)
    for seed in (1, 2):
        q = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((70, h), generator=q).bfloat16())
        logits.copy_(torch.randn((70, e), generator=q))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run(x, logits))
    want = run(x, logits)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(run(x, logits))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_grouped_positions_past_the_activations(bq):
    """Without rows a position is its activation row: those past the last count as zeros (their bias stays)."""
    g = torch.Generator().manual_seed(16)
    a, sa = codes((50, 256), g, 1)
    w, sw = codes((2, 256, 256), g, 128)
    bias = torch.randn((2, 256), generator=g).cuda()
    for p in (70, 300):
        off = torch.tensor([0, 20, p], dtype=torch.int32, device="cuda")
        out = bq.api.fp8_grouped_gemm(a, sa, off, w, sw, None, bias, out=torch.empty((p, 256), device="cuda"))
        ref = bq.api.fp8_grouped_gemm(a, sa, torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda"), w, sw, None, bias, out_dtype=F32)
        assert torch.equal(out[:50], ref) and torch.equal(out[50:], bias[1].expand(p - 50, 256))


@pytest.mark.parametrize("m,n,k", [(16, 7168, 2048), (100, 4096, 1152), (3, 2048, 1024), (40, 128, 512), (130, 1000, 640), (128, 136, 5120)])
def test_epilogue_shared_tiles(bq, m, n, k):
    """Products of few tiles, whose k-blocks two or four CTAs share; the same bits every time."""
    g = torch.Generator().manual_seed(m * n)
    a, sa = codes((m, k), g, 1)
    w, sw = codes((n, k), g, 128)
    bias = torch.randn(n, generator=g).cuda()
    res = torch.randn((m, n), generator=g).cuda()
    z, d = product(values(a, sa, 1), values(w, sw, 128), k // 128)
    # Up to four partial sums are joined: three more roundings of sums no larger than the bound's T / 2^-16.
    z = z + bias.double()
    d = d * (1 + 2.0 ** -6) + 2.0 ** -24 * (z.abs() + d)
    v, dv = after_act(z, d, "gelu_tanh")
    v = v + res.double()
    dv = dv + 2.0 ** -24 * (v.abs() + dv)
    got = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, "gelu_tanh", res, F32)
    bound_check(got, v, dv, F32, f"{m}x{n}x{k}")
    for _ in range(3):
        assert torch.equal(bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, "gelu_tanh", res, F32), got)


def test_products_of_unaligned_scales_and_odd_k_blocks(bq):
    """Scales that do not start on 16 bytes, and numbers of k-blocks that are no multiple of the stages'."""
    g = torch.Generator().manual_seed(18)
    for k in (128, 384, 640, 896, 1152):
        for m, n in ((5, 300), (200, 4096), (1500, 1600)):
            a, sa = codes((m, k), g, 1)
            w, sw = codes((n, k), g, 128)
            off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)   # noqa: E731
            want = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, None, "silu")
            assert torch.equal(bq.api.fp8_block_gemm_epilogue(a, off(sa), w, off(sw), None, "silu"), want)
            z, d = product(values(a, sa, 1), values(w, sw, 128), k // 128)
            bound_check(want, *after_act(z, d * (1 + 2.0 ** -6), "silu"), BF, f"{m}x{n}x{k}")


def test_training_step_of_a_dense_layer(bq):
    """Forward with the kept value before the activation, its gradient, and the product of the gradient's codes with the
    transposed weight: against the same steps in 64 bits on the same codes."""
    g = torch.Generator().manual_seed(19)
    m, n, k = 300, 512, 384
    a, sa = codes((m, k), g, 1)
    w, sw = codes((n, k), g, 128)
    bias = (0.1 * torch.randn(n, generator=g)).cuda()
    c, pre = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, "gelu", out_dtype=BF, save_pre=True)
    dy = torch.randn((m, n), generator=g).bfloat16().cuda()
    dz, db = bq.api.gemm_epilogue_backward(dy, pre, "gelu")
    z = pre.double().requires_grad_(True)
    act64(z, "gelu").backward(dy.double())
    assert ((db.double() - z.grad.sum(0)).abs() <= (2.0 ** -18 + m * 2.0 ** -24) * (dy.double().abs() * (2 + pre.double().abs())).sum(0)).all()
    ez, sz = bq.api.fp8_block_quantize(dz, 1, 128)
    wt, swt = w.t().contiguous(), sw.t().contiguous()
    da = bq.api.fp8_block_gemm_epilogue(ez, sz, wt, swt, out_dtype=F32)
    ref, err = product(values(ez, sz, 1), values(wt, swt, 128), n // 128)
    bound_check(da, ref, err * (1 + 2.0 ** -6), F32, "da")


def test_layer_of_no_tokens_and_of_no_local_expert(bq):
    g = torch.Generator().manual_seed(20)
    w1, s1 = codes((4, 512, 256), g, 128)
    w2, s2 = codes((4, 256, 256), g, 128)
    none = bq.api.fp8_moe(torch.empty((0, 256), dtype=BF, device="cuda"), torch.empty((0, 16), device="cuda"), w1, s1, w2, s2, 2)
    assert none.shape == (0, 256)
    x = torch.randn((9, 256), generator=g).bfloat16().cuda()
    logits = torch.full((9, 16), -5.0)
    logits[:, :4] = torch.randn((9, 4), generator=g)          # every choice is one of the first four experts
    res = torch.randn((9, 256), generator=g).bfloat16().cuda()
    out = bq.api.fp8_moe(x, logits.cuda(), w1, s1, w2, s2, 2, first_expert=8, residual=res)
    assert torch.equal(out, res)


def test_products_past_2_31_elements(bq):
    """Offsets of c, of the epilogue's tensors and of gathered rows that pass 32 bits: the last rows against a small call."""
    g = torch.Generator().manual_seed(21)
    p, n, k = 290_000, 8192, 128                              # c: 2.4e9 elements
    a, sa = codes((64, k), g, 1)
    w, sw = codes((2, n, k), g, 128)
    rows = (torch.arange(p, dtype=torch.int32) % 64).cuda()
    off = torch.tensor([0, 5, p], dtype=torch.int32, device="cuda")
    c = bq.api.fp8_grouped_gemm(a, sa, off, w, sw, rows, act="silu", out_dtype=BF)
    tail = bq.api.fp8_grouped_gemm(a, sa, torch.tensor([0, 0, 600], dtype=torch.int32, device="cuda"), w, sw, rows[-600:].contiguous(), act="silu")
    assert torch.equal(c[-600:], tail) and torch.equal(c[5 + 64 * 1000:5 + 64 * 1000 + 64], c[5:69])
    dz, db = bq.api.gemm_epilogue_backward(c, c, "silu")
    small, _ = bq.api.gemm_epilogue_backward(c[-600:].contiguous(), c[-600:].contiguous(), "silu")
    assert torch.equal(dz[-600:], small) and torch.isfinite(db).all()


def test_dense_product_past_2_31_elements(bq):
    g = torch.Generator().manual_seed(22)
    m, n, k = 290_000, 8192, 128
    a, sa = codes((m, k), g, 1)
    w, sw = codes((n, k), g, 128)
    bias = torch.randn(n, generator=g).cuda()
    c = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, "relu", out_dtype=BF)
    tail = bq.api.fp8_block_gemm_epilogue(a[-1000:].contiguous(), sa[-1000:].contiguous(), w, sw, bias, "relu", out_dtype=BF)
    assert torch.equal(c[-1000:], tail)


@pytest.mark.parametrize("counts", [[1, 0, 2], [5], [0, 3, 1, 1, 8, 0, 2, 9]])
@pytest.mark.parametrize("n", [1, 37, 130, 259])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_few_rows_odd_widths(bq, counts, n, gather):
    """Tiles of 32 rows in the form for widths that are no multiple of 8."""
    g = torch.Generator().manual_seed(n)
    off, offsets = offsets_of(counts)
    p = off[-1]
    a, sa = codes((p, 640), g, 1)
    w, sw = codes((len(counts), n, 640), g, 128)
    rows = torch.randint(0, p, (p,), generator=g).to(torch.int32).cuda() if gather else None
    bias = torch.randn((len(counts), n), generator=g).to(HF).cuda()
    for out in (BF, HF, F32):
        c = bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, rows, bias, "silu", out_dtype=out)
        bound_check(c, *grouped_ref(a, sa, rows, off, w, sw, bias, "silu", False), out, f"{n}")


@pytest.mark.parametrize("m,n,k", [(7, 361, 1152), (100, 129, 2048), (1, 2047, 1024), (128, 1022, 3200)])
def test_epilogue_shared_tiles_odd_widths(bq, m, n, k):
    g = torch.Generator().manual_seed(m + n)
    a, sa = codes((m, k), g, 1)
    w, sw = codes((n, k), g, 128)
    res = torch.randn((m, n), generator=g).to(HF).cuda()
    bias = torch.randn(n, generator=g).to(BF).cuda()
    z, d = product(values(a, sa, 1), values(w, sw, 128), k // 128)
    z = z + bias.double()
    d = d * (1 + 2.0 ** -6) + 2.0 ** -24 * (z.abs() + d)       # as in test_epilogue_shared_tiles
    v, dv = after_act(z, d, "silu")
    got, pre = bq.api.fp8_block_gemm_epilogue(a, sa, w, sw, bias, "silu", res, HF, True)
    bound_check(pre, z, d, HF, "pre")
    bound_check(got, v + res.double(), dv + 2.0 ** -24 * ((v + res.double()).abs() + dv), HF, f"{m}x{n}x{k}")


@pytest.mark.parametrize("raw", [False, True])
def test_scratch_belongs_to_the_stream_that_uses_it(bq, raw):
    """A call given another stream, which is busy: what the current stream allocates and writes after the call
    returned is not the call's scratch."""
    g = torch.Generator().manual_seed(30)
    e, h = 8, 256
    w1, s1 = codes((e, 512, h), g, 128)
    w2, s2 = codes((e, h, 256), g, 128)
    x = torch.randn((300, h), generator=g).bfloat16().cuda()
    logits = torch.randn((300, e), generator=g).cuda()
    dy, pre = (torch.randn((2000, 320), generator=g).bfloat16().cuda() for _ in range(2))
    want = bq.api.fp8_moe(x, logits, w1, s1, w2, s2, 4)
    want_dz, want_db = bq.api.gemm_epilogue_backward(dy, pre, "silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    arg = s.cuda_stream if raw else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)                # some 50 ms
    out = bq.api.fp8_moe(x, logits, w1, s1, w2, s2, 4, stream=arg)
    dz, db = bq.api.gemm_epilogue_backward(dy, pre, "silu", stream=arg)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
            for n in (512, 4096, 8192, 70_000, 160_000, 400_000, 700_000, 1 << 20) for _ in range(20)]
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(dz, want_dz) and torch.equal(db, want_db)
    assert all(bool((t == 255).all()) for t in held)
