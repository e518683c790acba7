"""Host-side checks of the dense-epilogue and expert-layer entries: arguments
are refused with a status, or by the binding with an exception, before anything
is enqueued. No GPU is needed: no call gets past its checks."""

import pytest
import torch

P = 0x10000          # never dereferenced


@pytest.fixture(scope="module")
def B():
    import dequantize_absmax_reduce_b200 as m
    return m._bq


def _route(B, dtype=None, t=4, e=64, score=1, ng=8, tg=4, gt=2, k=8, logits=P, bias=None, ids=P, w=P):
    return B.lib.bq_moe_route(logits, B.BQ_F32 if dtype is None else dtype, t, e, bias, score, ng, tg, gt, k, 1, 1.0, ids, w, None)


def test_route_refusals(B):
    inv, uns, mis = B.BQ_ERR_INVALID_ARG, B.BQ_ERR_UNSUPPORTED, B.BQ_ERR_MISALIGNED
    assert _route(B, dtype=B.BQ_F64) == uns and _route(B, dtype=B.BQ_S8) == uns and _route(B, score=2) == uns
    for kw in ({"t": -1}, {"e": 0}, {"e": 1056}, {"k": 0}, {"k": 33}, {"ng": 0}, {"ng": 33, "e": 33 * 8}, {"ng": 7},
               {"tg": 0}, {"tg": 9}, {"gt": 0}, {"gt": 3}, {"k": 33, "tg": 4}, {"e": 64, "ng": 16, "tg": 1, "k": 5},
               {"t": 1 << 28}, {"logits": None}, {"ids": None}, {"w": None}):
        assert _route(B, **kw) == inv, kw
    for kw in ({"logits": P + 2}, {"bias": P + 2}, {"ids": P + 1}, {"w": P + 3}):
        assert _route(B, **kw) == mis, kw
    assert _route(B, t=0) == B.BQ_OK and _route(B, t=0, logits=None, ids=None, w=None) == B.BQ_OK


def test_route_backward_refusals(B):
    f = lambda dt=B.BQ_BF16, t=4, e=64, ids=P, g=P, sc=0, k=8, l=P, d=P: B.lib.bq_moe_route_backward(   # noqa: E731
        l, dt, t, e, ids, g, sc, k, 0, 1.0, d, None)
    assert f(dt=B.BQ_F64) == B.BQ_ERR_UNSUPPORTED and f(sc=3) == B.BQ_ERR_UNSUPPORTED
    for kw in ({"t": -1}, {"e": 0}, {"e": 1025}, {"k": 0}, {"k": 40}, {"ids": None}, {"g": None}, {"l": None}, {"d": None}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"l": P + 1}, {"d": P + 1}, {"ids": P + 2}, {"g": P + 2}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert f(t=0) == B.BQ_OK


def test_group_refusals(B):
    f = lambda ids=P, t=4, k=2, first=0, n=8, o=P, r=P, p=P: B.lib.bq_moe_group(ids, t, k, first, n, o, r, p, None)   # noqa: E731
    for kw in ({"t": -1}, {"k": 0}, {"first": -1}, {"n": 0}, {"n": 1025}, {"ids": None}, {"o": None}, {"r": None}, {"p": None},
               {"t": 1 << 30, "k": 4}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"ids": P + 1}, {"o": P + 2}, {"r": P + 2}, {"p": P + 2}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw


def test_combine_refusals(B):
    f = lambda y=P, dt=B.BQ_BF16, yr=8, h=16, pos=P, w=P, t=4, k=2, r=None, o=P, odt=B.BQ_BF16: B.lib.bq_moe_combine(   # noqa: E731
        y, dt, yr, h, pos, w, t, k, r, o, odt, None)
    assert f(dt=B.BQ_F64) == B.BQ_ERR_UNSUPPORTED and f(odt=B.BQ_U8) == B.BQ_ERR_UNSUPPORTED
    for kw in ({"yr": -1}, {"h": -1}, {"h": 1 << 31}, {"t": -1}, {"k": 0}, {"y": None}, {"pos": None}, {"w": None}, {"o": None}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"y": P + 1}, {"o": P + 1}, {"r": P + 1}, {"pos": P + 1}, {"w": P + 2}, {"odt": B.BQ_F32, "o": P + 2}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert f(t=0) == B.BQ_OK and f(h=0) == B.BQ_OK
    g = lambda d=P, y=P, dt=B.BQ_F16, yr=8, h=16, pos=P, w=P, t=4, k=2, dy=P, dw=P: B.lib.bq_moe_combine_backward(   # noqa: E731
        d, y, dt, yr, h, pos, w, t, k, dy, dw, None)
    assert g(dt=B.BQ_F64) == B.BQ_ERR_UNSUPPORTED
    for kw in ({"yr": -1}, {"h": -1}, {"t": -1}, {"k": 0}, {"k": 33}, {"d": None}, {"y": None}, {"pos": None}, {"w": None},
               {"dy": None}, {"dw": None}):
        assert g(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"d": P + 1}, {"y": P + 1}, {"dy": P + 1}, {"pos": P + 1}, {"w": P + 2}, {"dw": P + 2}):
        assert g(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert g(t=0) == B.BQ_OK


def test_grouped_gemm_refusals(B):
    def f(a=P, sa=P, ar=8, k=256, rows=P, off=P, e=4, p=8, w=P, sw=P, n=512, bias=None, bt=B.BQ_F32, act=0, gated=0, c=P,
          ct=B.BQ_BF16):
        return B.lib.bq_fp8_grouped_gemm(a, sa, ar, k, rows, off, e, p, w, sw, n, bias, bt, act, gated, c, ct, None)
    for kw in ({"ct": B.BQ_F64}, {"ct": B.BQ_E4M3}, {"bias": P, "bt": B.BQ_F64}, {"act": -1}, {"act": 5}):
        assert f(**kw) == B.BQ_ERR_UNSUPPORTED, kw
    for kw in ({"ar": -1}, {"p": -1}, {"n": -1}, {"k": 0}, {"k": 100}, {"k": 1 << 31}, {"e": 0}, {"e": 1025}, {"n": 1 << 30},
               {"p": 1 << 31}, {"ar": 1 << 31}, {"gated": 1, "n": 128}, {"gated": 1, "n": 640}, {"off": None}, {"w": None},
               {"sw": None}, {"c": None}, {"a": None}, {"sa": None}, {"ar": 0}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"a": P + 8}, {"w": P + 8}, {"c": P + 8}, {"sa": P + 2}, {"sw": P + 2}, {"rows": P + 2}, {"off": P + 2},
               {"bias": P + 2}, {"bias": P + 1, "bt": B.BQ_BF16}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert f(p=0) == B.BQ_OK and f(n=0) == B.BQ_OK


def test_epilogue_refusals(B):
    def f(a=P, sa=P, m=8, k=256, w=P, sw=P, n=512, bias=None, bt=B.BQ_F32, act=0, res=None, c=P, ct=B.BQ_BF16, pre=None):
        return B.lib.bq_fp8_block_gemm_epilogue(a, sa, m, k, w, sw, n, bias, bt, act, res, c, ct, pre, None)
    for kw in ({"ct": B.BQ_F64}, {"bias": P, "bt": B.BQ_S8}, {"act": 9}):
        assert f(**kw) == B.BQ_ERR_UNSUPPORTED, kw
    for kw in ({"m": -1}, {"n": -1}, {"k": 0}, {"k": 64}, {"m": 1 << 31}, {"n": 1 << 31}, {"a": None}, {"sa": None}, {"w": None},
               {"sw": None}, {"c": None}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"a": P + 4}, {"w": P + 4}, {"c": P + 4}, {"res": P + 4}, {"pre": P + 4}, {"sa": P + 1}, {"sw": P + 1}, {"bias": P + 1}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert f(m=0) == B.BQ_OK and f(n=0) == B.BQ_OK
    ws = B.bq_gemm_epilogue_backward_workspace_size
    assert ws(0, 8) == 0 and ws(8, 0) == 0 and ws(-1, 8) == 0 and ws(1, 8) == 32 and ws(4096, 11008) % (4 * 11008) == 0
    g = lambda dy=P, pre=P, dt=B.BQ_BF16, m=8, n=16, act=4, dz=P, db=None, w=None, wb=0: B.lib.bq_gemm_epilogue_backward(   # noqa: E731
        dy, pre, dt, m, n, act, dz, db, w, wb, None)
    assert g(dt=B.BQ_F64) == B.BQ_ERR_UNSUPPORTED and g(act=7) == B.BQ_ERR_UNSUPPORTED
    for kw in ({"m": -1}, {"n": -1}, {"m": 1 << 31}, {"dy": None}, {"pre": None}, {"dz": None}, {"db": P}, {"db": P, "w": P, "wb": 63}):
        assert g(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"dy": P + 1}, {"pre": P + 1}, {"dz": P + 1}, {"db": P + 2, "w": P, "wb": 64}, {"db": P, "w": P + 2, "wb": 64}):
        assert g(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert g(n=0) == B.BQ_OK and g(m=0) == B.BQ_OK


def test_binding_checks_shapes_and_devices(B):
    """Tensors that do not fit together, or are not on a GPU, are refused before their pointers are taken."""
    import dequantize_absmax_reduce_b200 as bq
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        bq.api.moe_route(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        bq.api.moe_group(torch.zeros((4, 2), dtype=torch.int32), 8)
    need = B._need
    t = torch.zeros((4, 6), device="meta")
    for shape, dtypes in (((4, 7), (torch.float32,)), ((4,), (torch.float32,)), ((4, 6), (torch.float16,)), ((4, 6), (torch.float32,))):
        with pytest.raises(ValueError):
            need(t, "t", shape, dtypes, 0)
    with pytest.raises(ValueError, match="contiguous"):
        need(t.t(), "t", (6, 4), (torch.float32,), 0)
    assert need(None, "t", (1,), (torch.float32,), 0) is None


def test_scratch_of_the_default_stream(B, monkeypatch):
    """A stream given by its handle: 0 is the device's default stream (a wrapper around handle 0 would be another, new stream)."""
    import types

    import dequantize_absmax_reduce_b200 as bq
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    like = types.SimpleNamespace(is_cuda=True, device="cuda:3")
    assert bq.api._scratch_of(0, like) == ("default", "cuda:3")
    assert bq.api._scratch_of(0x5500, like) == ("external", 0x5500, "cuda:3")


def test_route_group_values(B):
    """BQ_GROUP_SCORES is a third way to value groups; numbers between are none."""
    assert _route(B, t=0, gt=B.BQ_GROUP_SCORES) == B.BQ_OK
    for gt in (B.BQ_GROUP_SCORES - 1, B.BQ_GROUP_SCORES + 1, -1):
        assert _route(B, t=0, gt=gt) == B.BQ_ERR_INVALID_ARG
    assert _route(B, gt=B.BQ_GROUP_SCORES, k=33) == B.BQ_ERR_INVALID_ARG


def test_combine_backward_whole_refusals(B):
    """As bq_moe_combine_backward, and its scratch (none for few rows and pairs)."""
    f = lambda d=P, y=P, dt=B.BQ_F16, yr=3000, h=16, pos=P, w=P, t=4, k=2, dy=P, dw=P, ws=P, wb=12000: (   # noqa: E731
        B.lib.bq_moe_combine_backward_whole(d, y, dt, yr, h, pos, w, t, k, dy, dw, ws, wb, None))
    assert f(dt=B.BQ_F64) == B.BQ_ERR_UNSUPPORTED
    for kw in ({"yr": -1}, {"yr": 1 << 31}, {"h": -1}, {"t": -1}, {"k": 0}, {"k": 33}, {"d": None}, {"y": None}, {"pos": None}, {"w": None},
               {"dy": None}, {"dw": None}, {"ws": None}, {"wb": 11999}, {"t": 0, "dy": None}, {"yr": 8, "ws": None, "dy": None}):
        assert f(**kw) == B.BQ_ERR_INVALID_ARG, kw
    for kw in ({"d": P + 1}, {"y": P + 1}, {"dy": P + 1}, {"pos": P + 1}, {"w": P + 2}, {"dw": P + 2}, {"ws": P + 2}):
        assert f(**kw) == B.BQ_ERR_MISALIGNED, kw
    assert f(t=0, yr=0) == B.BQ_OK and f(t=0, h=0) == B.BQ_OK
    size = B.bq_moe_combine_backward_workspace_size
    assert size(2048, 256, 8) == 0 and size(2049, 256, 8) == 8196 and size(8, 2049, 1) == 32
    assert size(0, 4, 2) == 0 and size(-1, 4, 2) == 0 and size(1 << 31, 4, 2) == 0 and size(3000, 0, 2) == 0 and size(3000, 4, 0) == 0
