"""Expert layers on the GPU: routing and its gradient, the expert order, the
combine step and its gradients, against plain definitions in 64 bits.

Tolerances, in units of u = 2^-24 (half a step of f32, relative):
  * weights: an exponential within 2 ulp (4 u), and at most eight more f32
    roundings through the score, the sum over at most 32 experts (5 levels) and
    the quotient: below 2^5 u = 2^-19 of the value;
  * logits' gradient: the same roundings on g and on sum g s, which may cancel:
    2^-18 of scale * s * (|g| + sum |g s|), plus the result's own half step;
  * combine: k + 1 fused steps of at most half a step of the running sum:
    (k + 2) u sum |w y| (+ the residual's), plus the result's half step;
  * dweights: products summed in f32 in any order: hidden * u * sum |d y|.
A half step of the result's type is eps / 2 relative, and half the smallest
subnormal where it is that small."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NEG = -math.inf


@pytest.fixture(scope="module")
def bq():
    import dequantize_absmax_reduce_b200 as m
    assert torch.cuda.is_available()
    return m


def half_step(t, dtype):
    fi = torch.finfo(dtype)
    return t.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- routing
def route_ref(x, top_k, bias, score, ng, tg, gt, renorm, scale):
    """Row by row in python floats (64 bits)."""
    ids, ws = [], []
    size = x.shape[1] // ng
    for row in x.double().tolist():
        bad = any(v != v for v in row)
        row = [NEG if v != v else v for v in row]
        if score == "sigmoid":
            s = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        else:
            top = max(row)
            e = [1.0 if v == top else math.exp(v - top) for v in row]
            s = [v / math.fsum(e) for v in e]
        v = list(row) if bias is None else [a + b for a, b in zip(s, bias.double().tolist())]
        v = [NEG if r == NEG or q != q else q for r, q in zip(row, v)]
        value = []
        for g in range(ng):
            best = sorted((q for q in v[g * size:(g + 1) * size] if q > NEG), reverse=True)[:gt]
            value.append(sum(best) if best else NEG)
        keep = sorted(range(ng), key=lambda g: (-value[g], g))[:tg]
        order = sorted((e for e in range(len(v)) if e // size in keep and v[e] > NEG), key=lambda e: (-v[e], e))[:top_k]
        d = math.fsum(s[e] for e in order) if renorm else 1.0
        w = [scale * s[e] / d if d > 0 else 0.0 for e in order]
        pad = top_k - len(order)
        ids.append(order + [-1] * pad)
        ws.append([math.nan] * top_k if bad else w + [0.0] * pad)
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(ws, dtype=torch.float64)


def check_route(bq, x, top_k, bias=None, score="sigmoid", ng=1, tg=1, gt=2, renorm=True, scale=1.0):
    ids, w = bq.api.moe_route(x.cuda(), top_k, None if bias is None else bias.cuda(), score, ng, tg, gt, renorm, scale)
    rid, rw = route_ref(x, top_k, bias, score, ng, tg, gt, renorm, scale)
    assert torch.equal(ids.cpu(), rid)
    w = w.cpu().double()
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    ok = torch.isnan(rw) | ((w - rw).abs() <= 2.0 ** -19 * rw.abs() + 2.0 ** -149)
    assert ok.all(), (w[~ok], rw[~ok])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,e,k,ng,tg,gt", [(1, 1, 1, 1, 1, 1), (7, 8, 2, 1, 1, 1), (33, 100, 5, 4, 2, 2), (64, 256, 8, 8, 4, 2),
                                            (50, 256, 8, 1, 1, 2), (9, 60, 6, 3, 2, 1), (5, 1024, 32, 32, 7, 2), (3, 513, 7, 27, 3, 2),
                                            (130, 160, 6, 8, 3, 1), (21, 384, 8, 1, 1, 1), (4, 64, 8, 32, 16, 2)])
def test_route(bq, score, with_bias, dtype, t, e, k, ng, tg, gt):
    g = gen(t + e + k)
    x = (1.5 * torch.randn((t, e), generator=g)).to(dtype)
    bias = 0.1 * torch.randn(e, generator=g) if with_bias else None
    check_route(bq, x, k, bias, score, ng, tg, gt, renorm=True, scale=2.5)
    check_route(bq, x, k, bias, score, ng, tg, gt, renorm=False, scale=1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_close_values(bq, score, with_bias):
    """Values that 32 bits cannot tell apart, and equal ones: the order is that
    of 64 bits, and of equal values the lowest index goes first."""
    g = gen(5)
    x = 2.0 + 1e-6 * torch.randn((200, 128), generator=g)
    x[:20] = 1.25
    x[20:40] = (4 * torch.randn((20, 128), generator=g)).round() / 4
    x[40:60, ::3] = x[40:60, 1:2]
    bias = torch.zeros(128) if with_bias else None
    if with_bias:
        bias[::2] = 1e-8
        bias[64:] = -0.25
    for ng, tg in ((1, 1), (8, 3)):
        check_route(bq, x, 8, bias, score, ng, tg, 2)
        check_route(bq, x, 8, bias, score, ng, tg, 1, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("ng,tg", [(1, 1), (4, 2)])
def test_route_masked_and_special(bq, score, with_bias, ng, tg):
    g = gen(9)
    x = torch.randn((16, 64), generator=g)
    x[0] = NEG                                   # nothing available
    x[1, 3:] = NEG                               # fewer than top_k
    x[2, :63] = NEG                              # one
    x[3, 5] = math.nan
    x[4] = math.nan
    x[5, 7] = math.inf
    x[6, 10] = x[6, 40] = math.inf
    x[7] = torch.finfo(torch.float32).min        # the type's lowest value is a logit like any other
    x[8, :16] = torch.finfo(torch.float32).min
    x[9] = 50.0
    x[10, ::2] = NEG
    x[11] = -90.0 + torch.randn(64, generator=g)
    bias = None
    if with_bias:
        bias = 0.1 * torch.randn(64, generator=g)
        bias[20], bias[21], bias[22] = NEG, math.nan, math.inf
    if score == "softmax":                       # the reference's shares of several infinite logits: see below
        inf = torch.isinf(x) & (x > 0)
        assert inf.sum() == 3
    for gt in (1, 2):
        check_route(bq, torch.where(x == math.inf, 60.0, x) if score == "softmax" else x, 6, bias, score, ng, tg, gt)
    if score == "softmax" and not with_bias and ng == 1:
        ids, w = bq.api.moe_route(x[5:7].cuda(), 2, None, "softmax", renormalize=False)
        assert ids.cpu()[:, 0].tolist() == [7, 10] and ids.cpu()[1, 1] == 40
        assert w.cpu()[0].tolist() == [1.0, 0.0] and w.cpu()[1].tolist() == [0.5, 0.5]


def test_route_small_sigmoid_scores_keep_their_ratio(bq):
    x = torch.full((2, 16), -300.0)
    x[0, 4], x[0, 9] = -200.0, -201.0
    x[1, 2] = 3.0
    ids, w = bq.api.moe_route(x.cuda(), 2, score="sigmoid")
    r = 1 / (1 + math.exp(-1.0))
    assert ids.cpu()[0].tolist() == [4, 9]
    assert (w.cpu()[0].double() - torch.tensor([r, 1 - r], dtype=torch.float64)).abs().max() < 2.0 ** -19


def test_route_many_rows_and_unaligned(bq):
    g = gen(11)
    x = torch.randn((5000, 64), generator=g)
    check_route(bq, x, 4, 0.05 * torch.randn(64, generator=g), "sigmoid", 8, 3, 2)
    buf = torch.randn(64 * 40 + 1, generator=g).cuda()
    v = buf[1:].view(40, 64)
    ids, w = bq.api.moe_route(v, 4)
    rid, _ = route_ref(v.cpu(), 4, None, "softmax", 1, 1, 2, True, 1.0)
    assert torch.equal(ids.cpu(), rid)
    assert bq.api.moe_route(x[:0].cuda(), 4)[0].shape == (0, 4)


def route_grad_ref(x, ids, g, score, renorm, scale):
    x = x.double().requires_grad_(True)
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, -1)
    there = ids >= 0
    c = torch.where(there, s.gather(1, ids.clamp_min(0).long()), 0.0)
    d = c.sum(-1, keepdim=True) if renorm else 1.0
    (scale * c / d * g.double()).sum().backward()
    cd, gd = c.detach(), g.double()
    spread = (gd.abs() * cd).sum(-1, keepdim=True) / (d.detach() if renorm else 1.0)
    weight = s.detach() / (d.detach() if renorm else 1.0)
    full = torch.zeros_like(weight).scatter_add_(1, ids.clamp_min(0).long(), torch.where(there, gd.abs(), 0.0))
    return x.grad, scale * weight * (full + spread)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,e,k", [(1, 8, 1), (17, 100, 5), (300, 128, 8), (31, 257, 32), (12, 1024, 8)])
def test_route_backward(bq, score, renorm, dtype, t, e, k):
    g = gen(t * e + k)
    x = (1.5 * torch.randn((t, e), generator=g)).to(dtype)
    ids = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(t)]).to(torch.int32)
    if k > 2:
        ids[::3, -1] = -1
    dw = torch.randn((t, k), generator=g)
    dx = bq.api.moe_route_backward(x.cuda(), ids.cuda(), dw.cuda(), score, renorm, 2.5).cpu()
    ref, size = route_grad_ref(x, ids, dw, score, renorm, 2.5)
    err = (dx.double() - ref).abs()
    assert (err <= 2.0 ** -18 * size + half_step(ref, dtype)).all(), err.max()
    if renorm or score == "sigmoid":             # nothing outside the chosen experts
        chosen = torch.zeros((t, e + 1), dtype=torch.bool).scatter_(1, torch.where(ids < 0, e, ids).long(), True)[:, :e]
        assert (dx[~chosen] == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(bq, score, renorm):
    """Central differences of the forward kernel's own weights."""
    g = gen(3)
    x = torch.randn((4, 16), generator=g)
    dw = torch.randn((4, 3), generator=g)
    ids, _ = bq.api.moe_route(x.cuda(), 3, None, score, renormalize=renorm)
    dx = bq.api.moe_route_backward(x.cuda(), ids, dw.cuda(), score, renorm).cpu().double()
    h = 2.0 ** -6
    for j in range(16):
        lo, hi = x.clone(), x.clone()
        lo[:, j] -= h
        hi[:, j] += h
        il, wl = bq.api.moe_route(lo.cuda(), 16, None, score, renormalize=False)
        ih, wh = bq.api.moe_route(hi.cuda(), 16, None, score, renormalize=False)
        loss = []
        for i, w in ((il, wl), (ih, wh)):
            s = torch.zeros((4, 16), dtype=torch.float64).scatter_(1, i.cpu().long(), w.cpu().double())
            c = s.gather(1, ids.cpu().long())
            loss.append(((c / c.sum(1, keepdim=True) if renorm else c) * dw.double()).sum(1))
        # Third derivatives of the weights are below 8 in size: h^2 / 6 * 8 * sum |dw|; weights to 2^-19 over 2h.
        bound = (h * h / 6 * 8 + 2.0 ** -18 / (2 * h)) * dw.abs().sum(1).double()
        assert (((loss[1] - loss[0]) / (2 * h) - dx[:, j]).abs() <= bound).all()


def test_route_backward_special_rows(bq):
    x = torch.randn((5, 16), generator=gen(1))
    x[0, 3:] = NEG
    x[1] = NEG
    x[2, 5] = math.nan
    ids = torch.tensor([[0, 1], [-1, -1], [0, 1], [4, 4], [2, 99]], dtype=torch.int32)
    dw = torch.ones((5, 2))
    dw[:, 1] = -0.5
    for score in ("sigmoid", "softmax"):
        for renorm in (False, True):
            dx = bq.api.moe_route_backward(x.cuda(), ids.cuda(), dw.cuda(), score, renorm).cpu()
            assert torch.isfinite(dx[[0, 3, 4]]).all()
            assert (dx[0, 3:] == 0).all()
            if score == "softmax" and not renorm:
                assert torch.isnan(dx[2]).all()
            else:
                assert (dx[1] == 0).all() and torch.isfinite(dx[2]).all()
            # The same index twice counts twice; an id past the experts has no weight.
            ref, size = route_grad_ref(x[3:4], ids[3:4], dw[3:4], score, renorm, 1.0)
            assert ((dx[3:4].double() - ref).abs() <= 2.0 ** -18 * size + 2.0 ** -24).all()
            one, size = route_grad_ref(x[4:5], torch.tensor([[2, -1]]), dw[4:5], score, renorm, 1.0)
            assert ((dx[4:5].double() - one).abs() <= 2.0 ** -18 * size + 2.0 ** -24).all()


# ---------------------------------------------------------------- expert order
def group_ref(ids, n, first):
    flat = ids.reshape(-1).tolist()
    k = ids.shape[1]
    lists = [[] for _ in range(n)]
    for i, e in enumerate(flat):
        if first <= e < first + n:
            lists[e - first].append(i)
    order = [i for l in lists for i in l]
    off = [0]
    for l in lists:
        off.append(off[-1] + len(l))
    pos = [-1] * len(flat)
    for p, i in enumerate(order):
        pos[i] = p
    rows = [i // k for i in order] + [-1] * (len(flat) - len(order))
    return off, rows, pos


@pytest.mark.parametrize("t,k,n,first", [(1, 1, 1, 0), (1, 8, 256, 0), (5, 3, 7, 2), (64, 8, 256, 0), (511, 8, 64, 64), (513, 8, 256, 0),
                                         (1000, 5, 1024, 0), (4096, 8, 32, 96), (3333, 3, 100, 0), (20000, 2, 8, 1)])
@pytest.mark.parametrize("kind", ["even", "skew", "one"])
def test_group(bq, t, k, n, first, kind):
    g = gen(t + k + n)
    e_all = n + 2 * first + 3
    if kind == "even":
        ids = torch.randint(-1, e_all, (t, k), generator=g)
    elif kind == "skew":
        ids = (torch.rand((t, k), generator=g) ** 4 * e_all).long()
    else:
        ids = torch.full((t, k), first + n - 1)
    ids = ids.to(torch.int32)
    off, rows, pos = bq.api.moe_group(ids.cuda(), n, first)
    ro, rr, rp = group_ref(ids, n, first)
    assert off.cpu().tolist() == ro and rows.cpu().tolist() == rr and pos.cpu().reshape(-1).tolist() == rp


def test_group_empty_and_outside(bq):
    off, rows, pos = bq.api.moe_group(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 5)
    assert off.cpu().tolist() == [0] * 6 and rows.numel() == 0 and pos.shape == (0, 4)
    ids = torch.tensor([[2 ** 31 - 1, -2 ** 31], [-1, 5]], dtype=torch.int32, device="cuda")
    off, rows, pos = bq.api.moe_group(ids, 5, 0)
    assert off.cpu().tolist() == [0] * 6 and (rows == -1).all() and (pos == -1).all()
    off, rows, pos = bq.api.moe_group(ids, 5, 2 ** 31 - 1)      # only the last id is one of these
    assert off.cpu().tolist() == [0, 1, 1, 1, 1, 1] and pos.cpu().tolist() == [[0, -1], [-1, -1]]


# ---------------------------------------------------------------- combine
def combine_case(t, k, h, dtype, seed, extra=3):
    g = gen(seed)
    p = t * k + extra
    pos = torch.randperm(p, generator=g)[:t * k].reshape(t, k).to(torch.int32)
    if t > 2:
        pos[1] = -1                               # a token none of whose experts is here
        pos[2, 0] = p + 5                         # past the rows
    return torch.randn((p, h), generator=g).to(dtype), pos, torch.rand((t, k), generator=g), g


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.float32, torch.float32),
                                       (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16), (torch.float16, torch.bfloat16)])
@pytest.mark.parametrize("t,k,h", [(1, 1, 1), (3, 2, 7), (5, 8, 64), (33, 6, 1000), (64, 8, 4096), (7, 40, 136), (130, 3, 72), (9, 5, 4100)])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(bq, dtype, out, t, k, h, residual):
    y, pos, w, g = combine_case(t, k, h, dtype, t + h)
    res = torch.randn((t, h), generator=g).to(out) if residual else None
    c = bq.api.moe_combine(y.cuda(), pos.cuda(), w.cuda(), None if res is None else res.cuda(), out).cpu()
    there = (pos >= 0) & (pos < y.shape[0])
    terms = torch.where(there, w, 0.0).double()[..., None] * y[torch.where(there, pos, 0).long()].double()
    ref, size = terms.sum(1), terms.abs().sum(1)
    if residual:
        ref, size = ref + res.double(), size + res.double().abs()
    err = (c.double() - ref).abs()
    assert c.dtype == out and (err <= (k + 2) * U * size + half_step(ref, out)).all(), err.max()


def test_combine_residual_in_place(bq):
    y, pos, w, g = combine_case(20, 4, 264, torch.bfloat16, 3)
    res = torch.randn((20, 264), generator=g).bfloat16().cuda()
    want = bq.api.moe_combine(y.cuda(), pos.cuda(), w.cuda(), res)
    bq._bq.bq_moe_combine(y.cuda(), pos.cuda(), w.cuda(), res, res)
    assert torch.equal(res, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("t,k,h", [(1, 1, 1), (3, 2, 7), (5, 8, 64), (33, 6, 1000), (64, 8, 4096), (9, 32, 136), (5, 3, 7168), (6, 2, 9001)])
def test_combine_backward(bq, dtype, t, k, h):
    y, pos, w, g = combine_case(t, k, h, dtype, t + h + 1)
    dout = torch.randn((t, h), generator=g).to(dtype)
    dy = torch.full_like(y, 7.0).cuda()
    dw = torch.empty((t, k), device="cuda")
    bq._bq.bq_moe_combine_backward(dout.cuda(), y.cuda(), pos.cuda(), w.cuda(), dy, dw)
    there = (pos >= 0) & (pos < y.shape[0])
    at = torch.where(there, pos, 0).long()
    ref = torch.full(y.shape, 7.0, dtype=torch.float64)            # rows that no position names stay
    ref[pos[there].long()] = (w.double()[..., None] * dout.double()[:, None, :])[there]
    err = (dy.cpu().double() - ref).abs()
    assert (err <= U * ref.abs() + half_step(ref * (1 + 2 * U), dtype)).all()
    terms = torch.where(there[..., None], y[at].double() * dout.double()[:, None, :], 0.0)
    assert ((dw.cpu().double() - terms.sum(-1)).abs() <= h * U * terms.abs().sum(-1)).all()
    a, b = bq.api.moe_combine_backward(dout.cuda(), y.cuda(), pos.cuda(), w.cuda())
    assert torch.equal(b, dw) and torch.equal(a[pos[there].long().cuda()], dy[pos[there].long().cuda()])


def test_unaligned_rows(bq):
    """Tensors that start off a 16-byte boundary take the kernels' scalar paths."""
    y, pos, w, g = combine_case(11, 4, 128, torch.bfloat16, 21)
    buf = torch.zeros(y.numel() + 1, dtype=torch.bfloat16, device="cuda")
    yu = buf[1:].view(y.shape)
    yu.copy_(y)
    assert torch.equal(bq.api.moe_combine(yu, pos.cuda(), w.cuda()), bq.api.moe_combine(y.cuda(), pos.cuda(), w.cuda()))
    dout = torch.randn((11, 128), generator=g).bfloat16().cuda()
    a, b = bq.api.moe_combine_backward(dout, yu, pos.cuda(), w.cuda())
    c, d = bq.api.moe_combine_backward(dout, y.cuda(), pos.cuda(), w.cuda())
    named = pos[(pos >= 0) & (pos < y.shape[0])].long().cuda()
    assert torch.equal(a[named], c[named])
    assert ((b - d).abs() <= 2 * 128 * U * 128 * 16).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e,ng,tg", [(256, 1, 1), (256, 8, 3), (60, 5, 2), (1024, 32, 9), (40, 1, 1)])
def test_route_clusters_of_near_values(bq, score, dtype, e, ng, tg):
    """Values in clusters far nearer than f32 scores can tell, of a few, of dozens and of more than a warp has lanes, astride
    the last place chosen; the same for groups' sums."""
    g = gen(e + ng)
    x = torch.randn((60, e), generator=g)
    for r in range(60):
        some = torch.randperm(e, generator=g)[:(3, 12, 30, min(e, 50))[r % 4]]
        x[r, some] = 3.0 + (1e-7 if r % 8 < 4 else 3e-6) * torch.randn(some.numel(), generator=g)
    bias = 1e-7 * torch.randn(e, generator=g)
    x = x.to(dtype)
    for k in (1, 5, min(8, e), min(32, tg * e // ng)):
        check_route(bq, x, k, bias, score, ng, tg, 2)
        check_route(bq, x, k, None, score, ng, tg, 2)
        check_route(bq, x, k, bias, score, ng, tg, 1)


def test_combine_without_rows(bq):
    """No expert's row is here: the residual alone, gradients of zero."""
    y = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[-1, 0], [3, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    res = torch.randn((2, 40), device="cuda").bfloat16()
    assert torch.equal(bq.api.moe_combine(y, pos, w, res), res)
    assert (bq.api.moe_combine(y, pos, w) == 0).all()
    dy, dw = bq.api.moe_combine_backward(res, y, pos, w)
    assert dy.shape == (0, 40) and (dw == 0).all()


def test_past_2_31_elements(bq):
    """Rows of y, dy and logits whose offsets pass 32 bits, against small calls on the same rows."""
    p, h = 290_000, 8192
    y = torch.randn((64, h), generator=gen(1)).bfloat16().cuda().repeat(p // 64 + 1, 1)[:p].contiguous()
    pos = torch.tensor([[p - 1, 0, p - 2], [p - 3, p - 4, -1]], dtype=torch.int32, device="cuda")
    w = torch.rand((2, 3), generator=gen(2)).cuda()
    at = pos.clamp_min(0).long()
    few, few_pos = y[at.reshape(-1)], torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3).where(pos >= 0, -1)
    assert torch.equal(bq.api.moe_combine(y, pos, w), bq.api.moe_combine(few, few_pos, w))
    dout = torch.randn((2, h), generator=gen(3)).bfloat16().cuda()
    dy, dw = bq.api.moe_combine_backward(dout, y, pos, w)
    dy2, dw2 = bq.api.moe_combine_backward(dout, few, few_pos, w)
    named = pos >= 0
    assert torch.equal(dw, dw2) and torch.equal(dy[pos[named].long()], dy2[few_pos[named].long()])
    del y, dy
    t, e = 2_200_000, 1024
    x = torch.randn((4096, e), generator=gen(4)).bfloat16().cuda().repeat(t // 4096 + 1, 1)[:t].contiguous()
    ids, wt = bq.api.moe_route(x, 4)
    i2, w2 = bq.api.moe_route(x[-5000:].contiguous(), 4)
    assert torch.equal(ids[-5000:], i2) and torch.equal(wt[-5000:], w2)
    dx = bq.api.moe_route_backward(x, ids, wt, renormalize=False)
    assert torch.equal(dx[-5000:], bq.api.moe_route_backward(x[-5000:].contiguous(), i2, w2, renormalize=False))


def test_order_of_many_pairs(bq):
    """More pairs than the warps of a cluster hold at once; many equal ids."""
    ids = torch.randint(-2, 70, (400_000, 6), generator=gen(5)).to(torch.int32)
    off, rows, pos = (v.cpu() for v in bq.api.moe_group(ids.cuda(), 64))
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < 64), flat, 64)
    order = torch.argsort(key, stable=True)
    n = int((key < 64).sum())
    assert off.tolist() == [0] + torch.bincount(key, minlength=65)[:64].cumsum(0).tolist()
    assert torch.equal(rows[:n].long(), order[:n] // 6) and (rows[n:] == -1).all()
    rank = torch.full_like(order, -1)
    rank[order[:n]] = torch.arange(n)
    assert torch.equal(pos.reshape(-1).long(), rank)
