"""Argument checks of the 128-block 8-bit entry points and of the few-token
forward: every case returns on the host before the first HIP call."""
import ctypes
import threading

import pytest
import torch

from sparse_moe_layer_04_amd import ops

ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_ALIGN = -1, -2, -3, -4, -5, -6
FAKE = 0x10000  # an aligned non-NULL address; never dereferenced (checks fail first)


@pytest.fixture(scope="module")
def L():
    return ops.lib()


def test_quantize_rows(L):
    def q(a=FAKE, dt=0, rows=4, K=128, codes=FAKE, scales=FAKE):
        return L.moe_quantize_fp8_block(a, dt, rows, K, codes, scales, None)
    assert q(rows=-1) == ERR_SHAPE
    assert q(K=0) == ERR_SHAPE
    assert q(rows=1 << 31, K=16) == ERR_SHAPE           # 2^31 blocks
    assert q(rows=1 << 40, K=16) == ERR_SHAPE
    assert q(K=120) == ERR_UNSUPPORTED
    assert q(dt=2) == ERR_UNSUPPORTED
    assert q(a=None) == ERR_NULL
    assert q(codes=None) == ERR_NULL
    assert q(scales=None) == ERR_NULL
    assert q(a=FAKE + 8) == ERR_ALIGN
    assert q(codes=FAKE + 4) == ERR_ALIGN
    assert q(scales=FAKE + 2) == ERR_ALIGN
    assert q(rows=0, a=None, codes=None, scales=None) == 0


def test_quantize_matrix(L):
    def q(w=FAKE, dt=0, G=2, N=100, K=128, codes=FAKE, scales=FAKE):
        return L.moe_quantize_weights_fp8_block(w, dt, G, N, K, codes, scales, None)
    assert q(G=0) == ERR_SHAPE
    assert q(N=0) == ERR_SHAPE
    assert q(K=0) == ERR_SHAPE
    assert q(G=1 << 20, N=1 << 20, K=1 << 20) == ERR_SHAPE
    assert q(N=(1 << 31) - 1, K=1 << 30) == ERR_SHAPE
    assert q(K=24) == ERR_UNSUPPORTED
    assert q(dt=-1) == ERR_UNSUPPORTED
    assert q(w=None) == ERR_NULL
    assert q(codes=FAKE + 1) == ERR_ALIGN


def test_grouped_gemm(L):
    def gg(a=FAKE, sa=FAKE, off=FAKE, G=2, rows=8, K=128, N=256, w=FAKE, sw=FAKE, dt=0, out=FAKE):
        return L.moe_grouped_gemm_fp8_block(a, sa, off, G, rows, K, N, w, sw, dt, out, None)
    assert gg(G=0) == ERR_SHAPE
    assert gg(rows=-1) == ERR_SHAPE
    assert gg(K=8) == ERR_SHAPE
    assert gg(N=0) == ERR_SHAPE
    assert gg(G=5000) == ERR_UNSUPPORTED
    assert gg(K=72) == ERR_UNSUPPORTED
    assert gg(N=40) == ERR_UNSUPPORTED
    assert gg(K=(1 << 22) + 16) == ERR_UNSUPPORTED
    assert gg(N=(1 << 22) + 16) == ERR_UNSUPPORTED
    assert gg(rows=(1 << 31) - 1, K=1 << 22) == ERR_SHAPE
    assert gg(dt=2) == ERR_UNSUPPORTED
    for name in ("a", "sa", "off", "w", "sw", "out"):
        assert gg(**{name: None}) == ERR_NULL, name
    assert gg(a=FAKE + 8) == ERR_ALIGN
    assert gg(w=FAKE + 1) == ERR_ALIGN
    assert gg(out=FAKE + 4) == ERR_ALIGN
    assert gg(sa=FAKE + 2) == ERR_ALIGN
    assert gg(sw=FAKE + 2) == ERR_ALIGN
    assert gg(rows=0, a=None, out=None) == 0


def test_expert_ffn(L):
    names = ("a", "sa", "off", "wg", "sg", "wu", "su", "wd", "sd", "h", "hs", "y")

    def ffn(G=2, rows=8, d=128, F=80, lim=10.0, mode=0, dt=1, **kw):
        p = {n: kw.get(n, FAKE) for n in names}
        return L.moe_expert_ffn_fp8_block(p["a"], p["sa"], p["off"], G, rows, d, F, p["wg"],
                                          p["sg"], p["wu"], p["su"], p["wd"], p["sd"],
                                          ctypes.c_float(lim), mode, p["h"], p["hs"], dt, p["y"],
                                          None)
    assert ffn(G=0) == ERR_SHAPE
    assert ffn(rows=-1) == ERR_SHAPE
    assert ffn(F=8) == ERR_SHAPE
    assert ffn(d=100) == ERR_UNSUPPORTED
    assert ffn(F=72) == ERR_UNSUPPORTED
    assert ffn(G=4097) == ERR_UNSUPPORTED
    assert ffn(lim=0.0) == ERR_SHAPE
    assert ffn(lim=float("nan")) == ERR_SHAPE
    assert ffn(mode=2) == ERR_UNSUPPORTED
    assert ffn(dt=3) == ERR_UNSUPPORTED
    for n in names:
        assert ffn(**{n: None}) == ERR_NULL, n
    for n in ("a", "wg", "wu", "wd", "h", "y"):
        assert ffn(**{n: FAKE + 8}) == ERR_ALIGN, n
    for n in ("sa", "sg", "su", "sd", "hs"):
        assert ffn(**{n: FAKE + 2}) == ERR_ALIGN, n
    assert ffn(rows=0, a=None, y=None) == 0


def few_cfg(**kw):
    base = dict(T=8, d=128, E=8, k=2, F=64, F_shared=64, mode=0, n_bias=1, V=0, scale=1.0,
                clamp_limit=10.0, clamp_mode=0, out_dtype=0)
    base.update(kw)
    return ops.MoeCfg(**base)


MATS = ("w_g", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")
SCALES = ("w_gate_scale", "w_up_scale", "w_down_scale", "s_gate_scale", "s_up_scale",
          "s_down_scale")


def test_forward_few(L):
    need = L.moe_forward_few_workspace_size(ctypes.byref(few_cfg(T=64, k=8, E=16)))
    assert need > 0

    def few(c=None, packed=0, x=FAKE, y=FAKE, ws=FAKE, wsb=need, ids=None, **ptr):
        c = c or few_cfg()
        m = {n: FAKE for n in MATS + ("score_bias",)}
        if packed == ops.WEIGHTS_FP8_BLOCK:
            m.update({n: FAKE for n in SCALES})
        m.update(ptr)
        w = ops.MoeWeights(packed=packed, **m)
        return L.moe_forward_few(ctypes.byref(c), ctypes.byref(w), x, ids, None, y, None, None,
                                 None, None, ws, wsb, None)
    w = ops.MoeWeights(packed=0)
    assert L.moe_forward_few(None, ctypes.byref(w), FAKE, None, None, FAKE, None, None, None,
                             None, FAKE, need, None) == ERR_NULL
    assert L.moe_forward_few(ctypes.byref(few_cfg()), None, FAKE, None, None, FAKE, None, None,
                             None, None, FAKE, need, None) == ERR_NULL
    for kw, code in (({"T": -1}, ERR_SHAPE), ({"T": 65}, ERR_UNSUPPORTED), ({"E": 0}, ERR_SHAPE),
                     ({"E": 1025}, ERR_UNSUPPORTED), ({"k": 9, "E": 16}, ERR_UNSUPPORTED),
                     ({"k": 3, "E": 2}, ERR_UNSUPPORTED), ({"d": 96}, ERR_UNSUPPORTED),
                     ({"F": 32}, ERR_SHAPE), ({"F_shared": 32}, ERR_UNSUPPORTED),
                     ({"F_shared": -64}, ERR_SHAPE), ({"mode": 2}, ERR_UNSUPPORTED),
                     ({"out_dtype": 2}, ERR_UNSUPPORTED), ({"clamp_limit": 0.0}, ERR_SHAPE),
                     ({"clamp_limit": float("nan")}, ERR_SHAPE),
                     ({"clamp_mode": 2}, ERR_UNSUPPORTED), ({"scale": float("nan")}, ERR_SHAPE),
                     ({"n_bias": 3}, ERR_SHAPE), ({"d": (1 << 22) + 64}, ERR_UNSUPPORTED),
                     ({"T": 64, "k": 8, "d": 1 << 22}, ERR_SHAPE)):
        assert few(few_cfg(**kw)) == code, kw
    for packed in (1, 2, 3, 4, 6):
        assert few(packed=packed) == ERR_UNSUPPORTED
    for n in MATS:
        assert few(**{n: None}) == ERR_NULL, n
        assert few(**{n: FAKE + 8}) == ERR_ALIGN, n
    for n in SCALES:
        assert few(packed=5, **{n: None}) == ERR_NULL, n
        assert few(packed=5, **{n: FAKE + 2}) == ERR_ALIGN, n
    assert few(score_bias=None) == ERR_NULL
    assert few(x=None) == ERR_NULL
    assert few(x=FAKE + 2) == ERR_ALIGN
    assert few(y=None) == ERR_NULL
    assert few(ws=None) == ERR_NULL
    assert few(ws=FAKE + 16) == ERR_WORKSPACE
    own = L.moe_forward_few_workspace_size(ctypes.byref(few_cfg()))
    assert few(wsb=own - 1) == ERR_WORKSPACE
    hash_cfg = few_cfg(mode=1, V=16, n_bias=0)
    assert few(hash_cfg) == ERR_NULL                     # no ids
    assert few(hash_cfg, ids=FAKE) == ERR_NULL           # no table
    assert few(few_cfg(mode=1, V=0), ids=FAKE, tid2eid=FAKE) == ERR_SHAPE
    assert few(few_cfg(T=0), x=None, y=None, ws=None) == 0


def test_forward_few_workspace(L):
    size = lambda **kw: L.moe_forward_few_workspace_size(ctypes.byref(few_cfg(**kw)))  # noqa: E731
    assert size(T=1) <= size(T=8) <= size(T=64)
    assert size(T=65) == 0 and size(d=100) == 0 and size(E=0) == 0
    assert L.moe_forward_few_workspace_size(None) == 0


def test_forward_refuses_block_weights(L):
    """moe_forward has no path for them: an error, not a reading of the codes
    as bf16."""
    c = few_cfg()
    w = ops.MoeWeights(packed=ops.WEIGHTS_FP8_BLOCK, **{n: FAKE for n in MATS + SCALES})
    assert L.moe_forward(ctypes.byref(c), ctypes.byref(w), FAKE, None, None, FAKE, None, None,
                         None, None, FAKE, 1 << 30, None) == ERR_UNSUPPORTED


def test_binding_refuses_host_and_mistyped_tensors():
    a = torch.zeros((4, 128))
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.quantize_fp8_block(a)
    with pytest.raises(ops.MoeError, match="bfloat16 or float32"):
        ops.quantize_fp8_block(a.half())
    with pytest.raises(ops.MoeError, match="bfloat16 or float32"):
        ops.quantize_weights_fp8_block(a.double())
    with pytest.raises(ops.MoeError, match="2 or 3 dims"):
        ops.quantize_weights_fp8_block(a.view(-1))
    c = torch.zeros((4, 128), dtype=torch.uint8)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.grouped_gemm_fp8_block(c, a, a, c, a)
    with pytest.raises(ops.MoeError, match="device tensor"):
        ops.expert_ffn_fp8_block(c, a, a, (c, a), (c, a), (c, a))


class OneCall:
    """The library with moe_forward_few replaced: keeps the arguments, and runs
    `meanwhile` once before it reads the config, as another thread may while
    the library is entered without the interpreter's lock."""

    def __init__(self, L):
        self.lib, self.meanwhile, self.calls = L, None, []

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def moe_forward_few(self, cfg, weights, x, *args):
        run, self.meanwhile = self.meanwhile, None
        if run:
            run()
        self.calls.append((cfg._obj.T, x, args[-3], args[-2]))
        return 0


def few_layer(monkeypatch, L, T=33, **kw):
    fake = OneCall(L)
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "_need", lambda t, *a, **k: t)
    monkeypatch.setattr(ops, "_stream", lambda: 0)
    shapes = dict(w_g=(8, 128), w_gate=(8, 64, 128), w_up=(8, 64, 128), w_down=(8, 128, 64))
    w = {n: torch.zeros(s, dtype=torch.bfloat16) for n, s in shapes.items()}
    return fake, ops.MoeLayer(T, 128, 8, 2, 64, 0, w, **kw)


def test_forward_few_counts_of_two_threads(L, monkeypatch):
    """Each call's token count is its own, whatever other threads' calls of the
    same layer do before the library reads it."""
    fake, layer = few_layer(monkeypatch, L)
    rows = {t: torch.zeros((t, 128), dtype=torch.bfloat16) for t in (1, 33)}

    def other():
        th = threading.Thread(target=layer.forward_few, args=(rows[33],))
        th.start()
        th.join()
    fake.meanwhile = other
    layer.forward_few(rows[1])
    assert [c[0] for c in fake.calls] == [33, 1]
    assert [c[1] for c in fake.calls] == [rows[33].data_ptr(), rows[1].data_ptr()]
    # one workspace, there from the start and large enough for both
    assert len({c[2] for c in fake.calls}) == 1 and fake.calls[0][2] == layer.few_ws.data_ptr()
    assert fake.calls[0][3] >= L.moe_forward_few_workspace_size(
        ctypes.byref(few_cfg(T=33, F_shared=0)))


def test_forward_few_on_a_workspace_of_the_callers(L, monkeypatch):
    fake, layer = few_layer(monkeypatch, L)
    own = layer.few_workspace()
    layer.forward_few(torch.zeros((2, 128), dtype=torch.bfloat16), ws=own)
    assert fake.calls[0][2:] == (own.data_ptr(), own.numel())
    assert own.data_ptr() != layer.few_ws.data_ptr() and own.numel() == layer.few_ws.numel()


def test_forward_few_refuses_other_workspaces(L, monkeypatch):
    need = ops._need
    _, layer = few_layer(monkeypatch, L)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    monkeypatch.setattr(ops, "_need", lambda t, dt, name, *a, **k:
                        need(t, dt, name, *a, **k) if name == "ws" else t)
    with pytest.raises(ops.MoeError, match="ws must be a device tensor"):
        layer.forward_few(x, ws=torch.empty(layer.few_ws.numel(), dtype=torch.uint8))
