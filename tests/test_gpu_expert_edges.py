"""Edges of the expert layers and of the products' epilogues: infinities, values
that cancel or vanish, rows that nobody names, tails of the activations, the
default stream by its number; against definitions in 64 bits. Tolerances stand
beside each test, in units of u = 2^-24, half a step of f32."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def bq():
    import dequantize_absmax_reduce_b200 as m
    assert torch.cuda.is_available()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- the default stream by its number
def test_stream_zero_is_the_default_stream(bq):
    """stream=0, the default stream's handle: calls stay in the order of that stream's work."""
    g = gen(91)
    e, h = 8, 256
    w1, s1 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * 512, h), generator=g)).bfloat16().cuda(), 128)
    w2, s2 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * h, 256), generator=g)).bfloat16().cuda(), 128)
    weights = (w1.view(e, 512, h), s1.view(e, 4, 2), w2.view(e, h, 256), s2.view(e, 2, 2))
    new = torch.randn((300, h), generator=g).bfloat16().cuda()
    logits = torch.randn((300, e), generator=g).cuda()
    want = bq.api.fp8_moe(new, logits, *weights, 4)
    x = torch.zeros_like(new)
    bq.api.fp8_moe(x, logits, *weights, 4, stream=0)
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    torch.cuda._sleep(100_000_000)                    # some 50 ms, behind which x gets its values
    x.copy_(new)
    out = bq.api.fp8_moe(x, logits, *weights, 4, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- choice of groups
def chosen_in_64_bits(x, bias, score, ng, tg, top_k):
    """Ids by f64 choice values score + bias, groups by the sum of their two largest; the lowest index of equal ones."""
    x = x.double()
    v = (torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, -1)) + bias.double()
    groups = v.reshape(x.shape[0], ng, -1)
    value = torch.sort(groups, dim=-1, descending=True).values[..., :2].sum(-1)
    kept = torch.zeros_like(value, dtype=torch.bool)
    kept.scatter_(1, torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :tg], True)
    v = torch.where(kept[..., None], groups, -math.inf).reshape(x.shape)
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[:, :top_k].to(torch.int32)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("e,ng,tg,k", [(256, 8, 4, 8), (64, 32, 16, 8), (60, 5, 2, 4), (512, 16, 3, 6)])
@pytest.mark.parametrize("size", [10.0, 50.0, 1e3, 1e4])
def test_group_sums_that_cancel(bq, score, e, ng, tg, k, size):
    """A group's two best choice values of opposite sign, far larger than their sum: the groups that stay are those of f64
    sums all the same (where groups end with lanes, and where they do not)."""
    g = gen(e + ng + int(size))
    x = torch.randn((3000, e), generator=g)
    bias = torch.full((ng, e // ng), -3.0 * size)
    bias[:, 0], bias[:, 1] = size, -size
    bias = bias.reshape(-1) + 0.01 * torch.rand(e, generator=g)
    ids, _ = bq.api.moe_route(x.cuda(), k, bias.cuda(), score, ng, tg, 2)
    want = chosen_in_64_bits(x, bias, score, ng, tg, k)
    wrong = (ids.cpu() != want).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} rows of 3000"


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("e,ng,tg,k", [(256, 8, 4, 8), (64, 8, 3, 4), (60, 5, 2, 4), (1024, 32, 7, 32), (8, 4, 2, 2)])
def test_groups_without_a_bias_are_those_of_zero_biases(bq, score, dtype, e, ng, tg, k):
    """Groups go by sums of scores, whether a bias of zeros is given or none."""
    x = (1.5 * torch.randn((500, e), generator=gen(e + k))).to(dtype)
    x[3, : e // 2] = -math.inf
    x[4] = -math.inf
    x[5, 1:] = -math.inf
    x[6] = 0.5
    zeros = torch.zeros(e)
    for renorm in (True, False):
        ids, w = bq.api.moe_route(x.cuda(), k, score=score, n_groups=ng, top_groups=tg, renormalize=renorm)
        ids0, w0 = bq.api.moe_route(x.cuda(), k, zeros.cuda(), score, ng, tg, 2, renorm)
        assert torch.equal(ids, ids0) and torch.equal(w, w0)
    full = torch.isfinite(x.double()).all(1)
    assert torch.equal(ids.cpu()[full], chosen_in_64_bits(x[full], zeros, score, ng, tg, k))


def test_layer_without_a_bias_is_that_of_zero_biases(bq):
    g = gen(31)
    e, h = 16, 256
    x = torch.randn((200, h), generator=g).bfloat16().cuda()
    logits = (1.5 * torch.randn((200, e), generator=g)).cuda()
    w1, s1 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * 512, h), generator=g)).bfloat16().cuda(), 128)
    w2, s2 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * h, 256), generator=g)).bfloat16().cuda(), 128)
    weights = (w1.view(e, 512, h), s1.view(e, 4, 2), w2.view(e, h, 256), s2.view(e, 2, 2))
    for top in ({}, {"group_top": 1}, {"group_top": 2}):
        kw = {"score": "sigmoid", "n_groups": 4, "top_groups": 2, **top}
        assert torch.equal(bq.api.fp8_moe(x, logits, *weights, 4, **kw),
                           bq.api.fp8_moe(x, logits, *weights, 4, bias=torch.zeros(e, device="cuda"), **kw))


# ---------------------------------------------------------------- NaN logits
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 4, 8, 9, 40])
@pytest.mark.parametrize("h", [64, 7])
def test_nan_weight_without_a_row_is_seen(bq, dtype, k, h):
    """A NaN weight, which marks a row of NaN logits, makes its token NaN although the position names no row."""
    y = torch.ones((50, h), dtype=dtype, device="cuda")
    pos = torch.full((6, k), -1, dtype=torch.int32)
    w = torch.full((6, k), 0.25)
    pos[0], pos[1] = 3, 3
    w[1, -1] = math.nan
    w[2] = math.nan
    w[3, -1], pos[3, -1] = math.nan, 50
    w[4, 0] = math.inf                              # not a NaN: nothing to add, nothing added
    res = torch.ones((6, h), dtype=dtype, device="cuda")
    for r in (None, res):
        out = bq.api.moe_combine(y, pos.cuda(), w.cuda(), r).float().cpu()
        assert (out[0] == 0.25 * k + (r is not None)).all() and torch.isnan(out[1:4]).all()
        assert (out[4:] == (0 if r is None else 1)).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_layer_shows_a_token_of_nan_logits(bq, score):
    """One NaN logit or nothing but NaN: the token comes out as NaN on every GPU that holds some of the experts, padded
    tokens (-inf) as their residual."""
    g = gen(81)
    x = torch.randn((6, 256), generator=g).bfloat16().cuda()
    w1, s1 = bq.api.fp8_block_quantize((0.05 * torch.randn((8 * 512, 256), generator=g)).bfloat16().cuda(), 128)
    w2, s2 = bq.api.fp8_block_quantize((0.05 * torch.randn((8 * 256, 256), generator=g)).bfloat16().cuda(), 128)
    w1, s1, w2, s2 = w1.view(8, 512, 256), s1.view(8, 4, 2), w2.view(8, 256, 256), s2.view(8, 2, 2)
    logits = torch.randn((6, 8), generator=g)
    logits[1], logits[2], logits[4, 3] = math.nan, -math.inf, math.nan
    res = torch.randn((6, 256), generator=g).bfloat16().cuda()
    for a, b in ((0, 8), (0, 4), (4, 8)):
        out = bq.api.fp8_moe(x, logits.cuda(), w1[a:b], s1[a:b], w2[a:b], s2[a:b], 3, score=score, first_expert=a, residual=res)
        assert torch.isnan(out[[1, 4]]).all() and torch.equal(out[2], res[2]) and torch.isfinite(out[[0, 2, 3, 5]]).all()


def half_step(t, dtype):
    fi = torch.finfo(dtype)
    return t.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


# ---------------------------------------------------------------- gradient rows that nobody names
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("t,k,h,p", [(1, 1, 1, 5), (5, 3, 7, 40), (33, 6, 1000, 500), (64, 8, 4096, 700), (9, 32, 136, 288), (0, 4, 64, 37),
                                     (6, 2, 9001, 100), (20, 2, 66, 3000), (700, 4, 24, 2900), (512, 4, 40, 2048), (513, 4, 40, 2052), (0, 3, 40, 2500)])
@pytest.mark.parametrize("stream", [None, "other", "raw"])
def test_combine_backward_returns_no_unwritten_row(bq, dtype, t, k, h, p, stream):
    """Rows of the returned gradient that no position names are zeros: memory that held NaN before is handed out."""
    g = gen(t + k + h)
    pos = torch.randperm(p, generator=g)[:t * k].reshape(t, k).to(torch.int32)
    if t > 2:
        pos[1], pos[2, 0], pos[2, -1] = -1, p, 2 ** 31 - 1
    y = torch.randn((p, h), generator=g).to(dtype).cuda()
    w = torch.rand((t, k), generator=g)
    dout = torch.randn((t, h), generator=g).to(dtype)
    s = None if stream is None else torch.cuda.Stream()
    args = [v.cuda() for v in (dout, pos, w)]
    torch.cuda.synchronize()
    for _ in range(4):
        held = [torch.full((p, h), math.nan, dtype=dtype, device="cuda"), torch.full((p,), 0, dtype=torch.int32, device="cuda")]
        torch.cuda.synchronize()
        del held
        dy, dw = bq.api.moe_combine_backward(args[0], y, args[1], args[2], stream=s.cuda_stream if stream == "raw" else s)
        torch.cuda.synchronize()
        there = (pos >= 0) & (pos < p)
        named = torch.zeros(p, dtype=torch.bool)
        named[pos[there].long()] = True
        assert (dy.cpu()[~named] == 0).all()
        ref = torch.zeros((p, h), dtype=torch.float64)
        ref[pos[there].long()] = (w.double()[..., None] * dout.double()[:, None, :])[there]
        assert ((dy.cpu().double() - ref).abs() <= U * ref.abs() + half_step(ref * (1 + 2 * U), dtype)).all()
        assert dw.shape == w.shape and (dw.cpu()[~there] == 0).all()


@pytest.mark.parametrize("t", [300, 900])
def test_combine_backward_of_some_experts_in_a_graph(bq, t):
    """Positions of a quarter of the experts, as the order gives them; captured once, replayed on another choice."""
    g = gen(41)
    k, h, e = 4, 264, 32
    ids = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(t)]).to(torch.int32).cuda()
    y, dout = torch.randn((t * k, h), generator=g).bfloat16().cuda(), torch.randn((t, h), generator=g).bfloat16().cuda()
    w = torch.rand((t, k), generator=g).cuda()

    def step():
        _, rows, pos = bq.api.moe_group(ids, 8, 8)
        return rows, pos, *bq.api.moe_combine_backward(dout, y, pos, w)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows, pos, dy, dw = step()
    for seed in (1, 2, 3):
        q = gen(seed)
        ids.copy_(torch.stack([torch.randperm(e, generator=q)[:k] for _ in range(t)]).to(torch.int32))
        dy.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        behind = rows < 0
        assert behind.any() and (dy[behind] == 0).all() and torch.isfinite(dy).all()
        n, named = int((~behind).sum()), pos >= 0
        want = torch.zeros((n, h), device="cuda")
        want[pos[named].long()] = (w[..., None] * dout.float()[:, None, :])[named]
        assert torch.equal(dy[:n], want.bfloat16())


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def biases_alone(bq, z, act, out, save_pre=False):
    """The dense epilogue of a product of zeros: its value before the activation is the bias."""
    a = torch.zeros((1, 128), dtype=torch.uint8, device="cuda")
    w = torch.zeros((z.numel(), 128), dtype=torch.uint8, device="cuda")
    sw = torch.ones(((z.numel() + 127) // 128, 1), device="cuda")
    return bq.api.fp8_block_gemm_epilogue(a, torch.ones((1, 1), device="cuda"), w, sw, z.cuda(), act, out_dtype=out, save_pre=save_pre)


# ---------------------------------------------------------------- slopes at infinity
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("n", [8, 3])
def test_slope_of_infinite_and_nan_values(bq, act, dtype, n):
    """The limits of the slopes, 1 and 0, to the last bit; a NaN stays one."""
    pre = torch.zeros((4, n), dtype=dtype, device="cuda")
    pre[0], pre[1], pre[2] = math.inf, -math.inf, math.nan
    dy = torch.full((4, n), 2.0, dtype=dtype, device="cuda")
    dz, db = bq.api.gemm_epilogue_backward(dy, pre, act)
    assert (dz[0] == 2).all() and (dz[1] == (2 if act == "none" else 0)).all()
    assert act == "none" or torch.isnan(dz[2]).all()
    _, db = bq.api.gemm_epilogue_backward(dy[:2].contiguous(), pre[:2].contiguous(), act)
    assert (db == (4 if act == "none" else 2)).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_kept_value_past_the_types_range(bq, act):
    """f16 keeps a value before the activation below -65504 as -inf, after which the activation is 0: so is its gradient."""
    z = torch.full((64,), -1e5)
    z[::2] = 1.0
    c, pre = biases_alone(bq, z, act, HF, True)
    assert (pre[0, 1::2] == -math.inf).all() and (c[0, 1::2] == 0).all()
    dz, db = bq.api.gemm_epilogue_backward(torch.ones_like(c), pre, act)
    assert (dz[0, 1::2] == 0).all() and (db[1::2] == 0).all() and torch.isfinite(dz).all() and torch.isfinite(db).all()


# ---------------------------------------------------------------- tails of the activations
def act_and_bound(z, act):
    """act(z) in 64 bits and the relative error of its f32 evaluation, from the formulas used.
    An argument's relative error d becomes |x| d of exp(x), and (2 y^2 + 1) d of erfc(y).
      * gelu, max(z, 0) - |z| Phi(-|z|): the exponent z^2 / 2 has a square, a constant and a product (3 u of it), ex2 within
        2^-22 (4 u), the factor beside it 10 u, three products: u (1.5 z^2 + 17);
      * silu, z / (1 + exp(-z)): constant and product of the exponent (2 u |z|), ex2 within 2^-22 (4 u), the sum (1 u), the
        reciprocal (2 u), the product (1 u): u (2 |z| + 8);
      * gelu (tanh), the same on the argument 2a: z^2, two constants, a fused step and a product: u (5 |2a| + 8)."""
    z = z.double()
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0)), U * (1.5 * z * z + 17)
    if act == "silu":
        return z * torch.sigmoid(z), U * (2 * z.abs() + 8)
    a2 = 2 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(a2), U * (5 * a2.abs() + 8)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", [F32, BF, HF])
def test_tails_of_the_activations(bq, act, out):
    """Relative to the value itself, where it is 1e-30 too; what lies below f32's normal numbers may be taken as 0."""
    z = torch.linspace(-30.0, 10.0, 20000)
    v, rel = act_and_bound(z, act)
    got = biases_alone(bq, z, act, out).cpu().double()[0]
    # Up to 2^-126 of the factor beside z is lost where it leaves the normal numbers.
    err = rel * (1 + 2.0 ** -10) * v.abs() + 2.0 ** -126 * z.double().abs()
    bad = (got - v).abs() > err + half_step(v.abs() + err, out)
    assert not bad.any(), (z[bad][:3], got[bad][:3], v[bad][:3])


def test_tail_of_the_gelu_slope(bq):
    """Phi(z) + z phi(z), relative to the two terms' sizes: Phi as in the forward pass (above 0 from 1, 2 u); phi the same
    exponential, u (1.5 z^2 + 4), a constant, two products and the last step."""
    z = torch.linspace(-30.0, 10.0, 20000)
    d = z.double()
    big, small = 0.5 * torch.erfc(-d / math.sqrt(2.0)), d * torch.exp(-0.5 * d * d) / math.sqrt(2.0 * math.pi)
    dz, _ = bq.api.gemm_epilogue_backward(torch.ones((1, z.numel()), device="cuda"), z.cuda()[None], "gelu")
    bound = U * (big * (1.5 * d * d + 18) + small.abs() * (1.5 * d * d + 8)) * (1 + 2.0 ** -10) + 2.0 ** -126 * (d.abs() + 1)
    bad = (dz.cpu().double()[0] - (big + small)).abs() > bound
    assert not bad.any(), (z[bad][:3], dz.cpu()[0][bad][:3], (big + small)[bad][:3])


# ---------------------------------------------------------------- gradients of the weights
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("e", [16, 100, 257])
def test_gradient_of_scores_that_vanish(bq, dtype, e):
    """Renormalised scores that 64 bits hold as zeros give weights of 0, whatever the logits: so their gradient is 0."""
    g = gen(e)
    bias = torch.zeros(e)
    bias[5], bias[6] = 11.0, 10.0
    near = -700.0 if dtype == F32 else -704.0
    for score, rest in (("sigmoid", -1000.0), ("softmax", 0.0)):
        x = torch.full((3, e), rest)
        x[:, 5], x[:, 6] = -900.0, -904.0
        x[1, 5], x[1, 6] = near, near - 4           # not vanished: shares of 1 / (1 + exp(-4)) and the rest
        x = x.to(dtype)
        ids, w = bq.api.moe_route(x.cuda(), 2, bias.cuda(), score)
        dw = torch.randn((3, 2), generator=g)
        dx = bq.api.moe_route_backward(x.cuda(), ids, dw.cuda(), score).cpu().double()
        assert ids.cpu().tolist() == [[5, 6]] * 3 and (w[[0, 2]] == 0).all() and (w[1] > 0).all()
        assert (dx[[0, 2]] == 0).all()
        r = 1 / (1 + math.exp(-4.0))
        ref = r * (1 - r) * (dw[1, 0] - dw[1, 1]).double()
        # g - sum and its product, 2^-18 of s (|g| + sum |g s|) as for every such gradient, and the result's half step
        size = r * 2 * dw[1].abs().sum().double()
        for at, want in ((5, ref), (6, -ref)):
            assert (dx[1, at] - want).abs() <= 2.0 ** -18 * size + half_step(want, dtype)


def test_dense_gradient_of_small_shares(bq):
    """Softmax as it is, chosen logits 60 to 87 below the largest: relative to their size. An exponential within 2 ulp (4 u)
    and its argument's rounding given back (1 u), the sum of 256 (8 u), reciprocal, and five products and sums: below 2^-19."""
    g = gen(61)
    x = -60.0 - 27.0 * torch.rand((400, 256), generator=g)
    x[:, 17] = torch.rand(400, generator=g)
    ids = torch.stack([torch.randperm(256, generator=g)[:6] for _ in range(400)]).to(torch.int32)
    dw = torch.randn((400, 6), generator=g)
    dx = bq.api.moe_route_backward(x.cuda(), ids.cuda(), dw.cuda(), "softmax", False).cpu().double()
    p = torch.softmax(x.double(), -1)
    full = torch.zeros_like(p).scatter_add_(1, ids.long(), dw.double())
    shift = (p * full).sum(-1, keepdim=True)
    size = p * (full.abs() + (p * full.abs()).sum(-1, keepdim=True))
    # (products with what is left of p below f32's normal numbers: 2^-149 a step, a few of them)
    assert ((dx - p * (full - shift)).abs() <= 2.0 ** -19 * size + 2.0 ** -146).all()


# ---------------------------------------------------------------- gathered rows on wide tiles
@pytest.mark.parametrize("counts", [[40], [17, 0, 130, 1, 90], [200, 129]])
@pytest.mark.parametrize("n,k", [(8, 128), (64, 384), (136, 1152), (512, 640)])
def test_grouped_gathered_rows_on_wide_tiles(bq, counts, n, k):
    """More than 16 gathered rows an expert, narrow and few weights, scales off 16-byte boundaries, rows outside the
    activations, positions behind the last: the sums are those of the dense product of each expert's rows, where one CTA
    sums all of k (bit for bit: the same blocks in the same order), and the same every time."""
    g = gen(n + k + sum(counts))
    e, p, t = len(counts), sum(counts), 70

    def codes(*shape):
        c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        return torch.where((c & 127) == 127, 0x38, c).to(torch.uint8).cuda()
    off16 = lambda v: torch.cat([v.new_zeros(1), v.reshape(-1)])[1:].view(v.shape)   # noqa: E731
    a, sa = codes(t, k), off16((torch.rand((t, k // 128), generator=g) * 0.01).cuda())
    w, sw = codes(e, n, k), off16((torch.rand((e, (n + 127) // 128, k // 128), generator=g) * 0.01).cuda())
    rows = torch.randint(0, t, (p + 5,), generator=g).to(torch.int32)
    rows[3], rows[9] = -1, t
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    out = torch.full((p + 5, n), 3.0, device="cuda")
    bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, rows.cuda(), act="silu", out=out)
    first = out.clone()
    for _ in range(3):
        bq.api.fp8_grouped_gemm(a, sa, offsets, w, sw, rows.cuda(), act="silu", out=out)
        assert torch.equal(out, first)
        assert (out[p:] == 3.0).all() and (out[[3, 9]] == 0).all()
        for i in range(e):
            mine = rows[at[i]:at[i + 1]].long()
            here = (mine >= 0) & (mine < t)
            if not here.any():
                continue
            x = mine[here].cuda()
            z = bq.api.fp8_block_gemm_quantized(a[x], sa[x], w[i], sw[i].clone(), F32)
            got = out[at[i]:at[i + 1]][here.cuda()].double()
            want, rel = act_and_bound(z, "silu")
            assert ((got - want).abs() <= rel * want.abs() + half_step(want, F32) + 2.0 ** -126 * z.double().abs()).all()
