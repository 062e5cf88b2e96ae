"""Argument checks of the norm, balance-loss, gradient-clipping and MXFP4 entry
points: every case returns on the host before the first HIP call."""
import ctypes

import pytest
import torch

from sparse_moe_layer_04_amd import ops

ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_ALIGN = -1, -2, -3, -4, -5, -6
FAKE = 0x10000  # an aligned non-NULL address; never dereferenced (checks fail first)
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return ops.lib()


def test_add_rms_norm(L):
    def f(x=FAKE, xt=0, res=FAKE, rt=0, w=FAKE, wt=0, rows=4, d=128, eps=1e-6, out=FAKE, y=FAKE,
          codes=FAKE, scales=FAKE):
        return L.moe_add_rms_norm(x, xt, res, rt, w, wt, rows, d, eps, out, y, codes, scales, None)
    assert f(rows=-1) == ERR_SHAPE
    assert f(rows=1 << 31) == ERR_SHAPE
    assert f(d=0) == ERR_SHAPE
    assert f(d=12) == ERR_UNSUPPORTED
    assert f(d=16392) == ERR_UNSUPPORTED
    assert f(d=24) == ERR_UNSUPPORTED                  # codes: a multiple of 16
    assert f(eps=-1e-6) == ERR_SHAPE
    assert f(eps=NAN) == ERR_SHAPE
    assert f(eps=INF) == ERR_SHAPE
    for n in ("xt", "rt", "wt"):
        assert f(**{n: 2}) == ERR_UNSUPPORTED, n
    assert f(x=None) == ERR_NULL
    assert f(w=None) == ERR_NULL
    assert f(out=None) == ERR_NULL                     # a residual needs its output
    assert f(codes=None) == ERR_NULL
    assert f(scales=None) == ERR_NULL
    assert f(y=None, codes=None, scales=None) == ERR_NULL
    for n in ("x", "res", "w", "out", "y", "codes"):
        assert f(**{n: FAKE + 8}) == ERR_ALIGN, n
    assert f(scales=FAKE + 2) == ERR_ALIGN
    assert f(rows=0, x=None, y=None) == 0


def test_rms_norm_backward(L):
    size = L.moe_rms_norm_backward_workspace_size
    assert size(-1, 128) == size(4, 0) == size(4, 12) == size(4, 16392) == 0
    assert size(0, 8) >= 32 and size(10 ** 6, 4096) >= 4096 * 4
    need = size(4, 128)

    def f(s=FAKE, st=0, w=FAKE, wt=0, dy=FAKE, gt=0, res=FAKE, rt=0, rows=4, d=128, eps=1e-6,
          dx=FAKE, xt=1, dw=FAKE, ws=FAKE, wsb=need):
        return L.moe_rms_norm_backward(s, st, w, wt, dy, gt, res, rt, rows, d, eps, dx, xt, dw, ws,
                                       wsb, None)
    assert f(rows=-1) == ERR_SHAPE
    assert f(d=12) == ERR_UNSUPPORTED
    assert f(eps=NAN) == ERR_SHAPE
    for n in ("st", "wt", "gt", "rt", "xt"):
        assert f(**{n: -1}) == ERR_UNSUPPORTED, n
    for n in ("s", "w", "dy", "dx", "dw", "ws"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("s", "w", "dy", "res", "dx", "dw"):
        assert f(**{n: FAKE + 4}) == ERR_ALIGN, n
    assert f(ws=FAKE + 128) == ERR_WORKSPACE
    assert f(wsb=need - 1) == ERR_WORKSPACE
    assert f(rows=0, s=None, dw=None) == ERR_NULL      # dw is written all the same


def test_balance_loss(L):
    size = L.moe_balance_loss_workspace_size
    assert size(-1, 8, 1, 1) == size(8, 0, 1, 1) == size(8, 8, 0, 1) == size(8, 8, 1, 3) == 0
    assert size(8, 1025, 1, 1) == size(8, 8, (1 << 20) + 1, 1) == 0
    assert size(0, 8, 1, 1) > 0
    need = size(64, 8, 3, 1)
    assert size(64, 8, 3, 2) > need

    def f(lg=FAKE, ids=FAKE, off=FAKE, mod=None, mask=None, T=64, E=8, k=2, S=3, loss=FAKE,
          counts=FAKE, ws=FAKE, wsb=need):
        return L.moe_balance_loss(lg, ids, off, mod, mask, T, E, k, S, loss, counts, None, ws, wsb,
                                  None)

    def b(lg=FAKE, ids=FAKE, off=FAKE, counts=FAKE, dl=FAKE, T=64, E=8, k=2, S=3, out=FAKE):
        return L.moe_balance_loss_backward(lg, ids, off, None, None, counts, dl, None, T, E, k, S,
                                           out, None)
    for g in (f, b):
        assert g(T=-1) == ERR_SHAPE
        assert g(E=0) == ERR_SHAPE
        assert g(k=0) == ERR_SHAPE
        assert g(S=0) == ERR_SHAPE
        assert g(T=1 << 30, k=2) == ERR_SHAPE
        assert g(E=1025) == ERR_UNSUPPORTED
        assert g(k=9) == ERR_UNSUPPORTED
        assert g(S=(1 << 20) + 1) == ERR_UNSUPPORTED
        assert g(off=None) == ERR_NULL                 # three sequences need offsets
        for n in ("lg", "ids", "counts"):
            assert g(**{n: None}) == ERR_NULL, n
    assert f(loss=None) == ERR_NULL
    assert f(ws=None) == ERR_NULL
    assert f(ws=FAKE + 64) == ERR_WORKSPACE
    assert f(wsb=need - 1) == ERR_WORKSPACE
    assert f(T=0, loss=None) == ERR_NULL               # the losses are written all the same
    assert b(dl=None) == ERR_NULL
    assert b(out=None) == ERR_NULL
    assert b(T=0, lg=None, out=None) == 0


def plan_of(L, tensors):
    e = (ops.MoeGradTensor * len(tensors))(*[ops.MoeGradTensor(*t) for t in tensors])
    n = L.moe_grad_plan_size(e, len(tensors))
    buf = (ctypes.c_uint8 * max(n, 1))()
    return L.moe_grad_plan(e, len(tensors), buf, n), bytes(buf)[:n]


def test_grad_plan(L):
    A = 1 << 20
    assert plan_of(L, [(A, A, 8193, 1)])[0] == 0
    st, p = plan_of(L, [(A, A, 8193, 1), (0, 0, 0, 0), (2 * A, 3 * A, 20000, 0)])
    assert st == 0 and len(p) == 32 * (2 + 3)
    at = [(int.from_bytes(p[i:i + 8], "little"), int.from_bytes(p[i + 8:i + 16], "little"),
           int.from_bytes(p[i + 16:i + 20], "little"), p[i + 20]) for i in range(0, len(p), 32)]
    assert at == [(A, A, 8192, 1), (A + 32768, A + 32768, 1, 1), (2 * A, 3 * A, 8192, 0),
                  (2 * A + 16384, 3 * A + 16384, 8192, 0),
                  (2 * A + 32768, 3 * A + 32768, 20000 - 16384, 0)]
    assert plan_of(L, [(A, A, -1, 1)])[0] == ERR_SHAPE
    assert plan_of(L, [(A, A, 8, 2)])[0] == ERR_UNSUPPORTED
    assert plan_of(L, [(None, A, 8, 1)])[0] == ERR_NULL
    assert plan_of(L, [(A, None, 8, 1)])[0] == ERR_NULL
    assert plan_of(L, [(A + 8, A + 8, 8, 1)])[0] == ERR_ALIGN
    assert plan_of(L, [(A, A + 4, 8, 1)])[0] == ERR_ALIGN
    # the same tensor twice, tensors that overlap, an out over another's gradient
    assert plan_of(L, [(A, A, 8, 1), (A, A, 8, 1)])[0] == ERR_UNSUPPORTED
    assert plan_of(L, [(A, A, 16, 1), (A + 48, A + 48, 8, 1)])[0] == ERR_UNSUPPORTED
    assert plan_of(L, [(A, A, 16, 0), (A + 32, A + 32, 8, 1)])[0] == 0
    assert plan_of(L, [(A, 2 * A, 8, 1), (3 * A, A, 8, 1)])[0] == ERR_UNSUPPORTED
    assert plan_of(L, [(A, A + 16, 8, 1)])[0] == ERR_UNSUPPORTED
    assert plan_of(L, [(A + 16, A, 8, 1)])[0] == ERR_UNSUPPORTED
    # one gradient read for two outs is no harm
    assert plan_of(L, [(A, 2 * A, 8, 1), (A, 3 * A, 8, 1)])[0] == 0
    e = (ops.MoeGradTensor * 1)(ops.MoeGradTensor(A, A, 8, 1))
    buf = (ctypes.c_uint8 * 64)()
    assert L.moe_grad_plan(e, 1, buf, 64) == ERR_SHAPE
    assert L.moe_grad_plan(e, 1, None, 32) == ERR_NULL
    assert L.moe_grad_plan(None, 1, buf, 32) == ERR_NULL
    assert L.moe_grad_plan(e, -1, buf, 0) == ERR_SHAPE
    assert L.moe_grad_plan_size(e, -1) == 0 and L.moe_grad_plan_size(None, 1) == 0


def test_grad_norm(L):
    def f(plan=FAKE, n=64, norm=FAKE, ws=FAKE, wsb=16384):
        return L.moe_grad_norm(plan, n, norm, ws, wsb, None)

    def c(max_norm=1.0, plan=FAKE, n=64, norm=FAKE, ws=FAKE, wsb=16384):
        return L.moe_clip_grad_norm(plan, n, max_norm, norm, ws, wsb, None)
    for g in (f, c):
        assert g(n=40) == ERR_SHAPE
        assert g(plan=None) == ERR_NULL
        assert g(norm=None) == ERR_NULL
        assert g(ws=None) == ERR_NULL
        assert g(ws=FAKE + 16) == ERR_WORKSPACE
        assert g(wsb=16383) == ERR_WORKSPACE
        assert g(plan=FAKE + 16) == ERR_ALIGN
        assert g(norm=FAKE + 2) == ERR_ALIGN
    assert c(max_norm=-1.0) == ERR_SHAPE
    assert c(max_norm=NAN) == ERR_SHAPE


def test_quantize_mxfp4(L):
    def q(a=FAKE, dt=0, rows=4, K=128, codes=FAKE, scales=FAKE):
        return L.moe_quantize_mxfp4(a, dt, rows, K, codes, scales, None)
    assert q(rows=-1) == ERR_SHAPE
    assert q(K=0) == ERR_SHAPE
    assert q(rows=1 << 62, K=1 << 30) == ERR_SHAPE
    assert q(K=48) == ERR_UNSUPPORTED
    assert q(dt=2) == ERR_UNSUPPORTED
    for n in ("a", "codes", "scales"):
        assert q(**{n: None}) == ERR_NULL, n
    assert q(a=FAKE + 8) == ERR_ALIGN
    assert q(codes=FAKE + 8) == ERR_ALIGN
    assert q(rows=0, a=None) == 0


def test_grouped_gemm_mxfp4(L):
    def gg(a=FAKE, sa=FAKE, off=FAKE, G=2, rows=8, K=128, N=256, w=FAKE, sw=FAKE, dt=0, out=FAKE):
        return L.moe_grouped_gemm_mxfp4(a, sa, off, G, rows, K, N, w, sw, dt, out, None)
    assert gg(G=0) == ERR_SHAPE
    assert gg(rows=-1) == ERR_SHAPE
    assert gg(K=16) == ERR_SHAPE
    assert gg(N=0) == ERR_SHAPE
    assert gg(G=5000) == ERR_UNSUPPORTED
    assert gg(K=80) == ERR_UNSUPPORTED
    assert gg(N=40) == ERR_UNSUPPORTED
    assert gg(K=(1 << 22) + 32) == ERR_UNSUPPORTED
    assert gg(N=(1 << 22) + 16) == ERR_UNSUPPORTED
    assert gg(rows=(1 << 31) - 1, K=1 << 22) == ERR_SHAPE
    assert gg(dt=2) == ERR_UNSUPPORTED
    for name in ("a", "sa", "off", "w", "sw", "out"):
        assert gg(**{name: None}) == ERR_NULL, name
    for name in ("a", "w", "out"):
        assert gg(**{name: FAKE + 8}) == ERR_ALIGN, name
    assert gg(rows=0, a=None, out=None) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 128), torch.ones(128)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.add_rms_norm(x, w)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.rms_norm_backward(x, w, x)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.balance_loss(x, ids)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.balance_loss_backward(x, ids, ids, x)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.GradClip([x])
    with pytest.raises(ops.MoeError, match="a tensor"):
        ops.GradClip([])
    with pytest.raises(ops.MoeError, match="out must hold 1"):
        ops.GradClip([x], out=[])
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.quantize_mxfp4(x)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.grouped_gemm_mxfp4(u8, u8, off, u8, u8)
    for call in (lambda: ops.add_rms_norm(None, w), lambda: ops.rms_norm_backward(None, w, x),
                 lambda: ops.balance_loss(None, ids), lambda: ops.quantize_mxfp4(None),
                 lambda: ops.GradClip([None]), lambda: ops.grouped_gemm_mxfp4(None, u8, off, u8, u8)):
        with pytest.raises(ops.MoeError, match="is required"):
            call()


@pytest.mark.parametrize("dx_dtype", [torch.float32, torch.bfloat16, 2, -1, None, "fp32"])
def test_binding_refuses_types_of_dx(dx_dtype):
    """What is neither OUT_F32 nor OUT_BF16 is no bf16 either."""
    x, w = torch.zeros(4, 128), torch.ones(128)
    with pytest.raises(ops.MoeError, match="dx_dtype"):
        ops.rms_norm_backward(x, w, x, dx_dtype=dx_dtype)
