"""The training example: a block's gradients against 64-bit autograd, and the
operators around the layer in one run.

The block rounds to bf16 what enters its matrix products on the way back (the
experts' output gradients, the pre-activations' gradients, h, the balance
loss's gradient in the logits): at most four roundings of half a step (2^-8) in
series, so a gradient is within 4 * 2^-8 of the reference's in the 2-norm.
What is rounded on the way forward (the stream, the normalised rows) is given
to the reference as it is.
"""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import training_step as example  # noqa: E402

from sparse_moe_layer_04_amd import ops, workloads  # noqa: E402

pytestmark = pytest.mark.gpu
D = torch.float64


def as_given(v, actual):
    """v's gradient, the values that were rounded."""
    return v + (actual.cpu().to(D) - v).detach()


def reference(block, x, stream, c_out, c_s):
    w, inp = block.w, {n: v.cpu() for n, v in block.inputs.items() if torch.is_tensor(v)}
    leaf = {n: inp[n].to(D).requires_grad_() for n in block.weights}
    leaf["norm"] = block.norm.cpu().to(D).requires_grad_()
    leaf["x"] = x.cpu().to(D).requires_grad_()
    s = as_given(leaf["x"] + stream.cpu().to(D), block.s)
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + block.eps)
    y = as_given(n * leaf["norm"], block.y)
    ids = block.ids.cpu().long()
    score = torch.sigmoid(y @ leaf["w_g"].t())
    g = score.gather(1, ids)
    wt = g / g.sum(1, keepdim=True) * w.scale

    def ffn(v, gate, up, down):
        a = (v @ gate.t()).clamp(-w.clamp_limit, w.clamp_limit)
        b = (v @ up.t()).clamp(-w.clamp_limit, w.clamp_limit)
        return (a * torch.sigmoid(a) * b) @ down.t()
    out = ffn(y, leaf["s_gate"], leaf["s_up"], leaf["s_down"]) if w.Fs else torch.zeros_like(y)
    for e in range(w.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            rows = ffn(y[t], leaf["w_gate"][e], leaf["w_up"][e], leaf["w_down"][e])
            out = out.index_add(0, t, rows * wt[t, j][:, None])
    # the balance losses with their weights
    p = score / score.sum(1, keepdim=True)
    mod = torch.zeros(w.T, dtype=torch.long) if block.modality is None else \
        (block.modality.cpu() != 0).long()
    total = (out * c_out.cpu().to(D)).sum() + (s * c_s.cpu().to(D)).sum()
    off = block.offsets.tolist()
    losses = torch.zeros(block.d_loss.shape, dtype=D)
    for i in range(len(off) - 1):
        for c in range(block.d_loss.shape[1]):
            t = torch.arange(off[i], off[i + 1])
            t = t[mod[t] == c]
            if not len(t):
                continue
            f = torch.bincount(ids[t].reshape(-1), minlength=w.E).to(D) * w.E / (w.k * len(t))
            loss = (p[t] @ f).mean()
            losses[i, c] = loss.detach()
            total = total + loss * float(block.d_loss[i, c])
    total.backward()
    return {n: v.grad for n, v in leaf.items()}, losses


@pytest.mark.parametrize("T,d,E,k,F,Fs,n_bias,rt", [
    (130, 256, 64, 4, 128, 128, 1, torch.bfloat16), (97, 192, 64, 6, 64, 0, 2, torch.float32)])
def test_gradients(T, d, E, k, F, Fs, n_bias, rt):
    w = workloads.small(T, d, E, k, F, 11, scale=2.5, F_shared=Fs, n_bias=n_bias)
    inputs = workloads.make_inputs(w, "cuda")
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    block = example.Block(w, inputs, off, balance=200.0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda: torch.randn((T, d), generator=gen, device="cuda")  # noqa: E731
    block.norm += 0.2 * torch.randn(d, generator=gen, device="cuda")
    x, stream, c_out, c_s = inputs["x"], rand().to(rt), rand(), rand()
    out, s, loss = block.forward(x, stream)
    assert s.dtype == rt and out.dtype == torch.float32
    dx = block.backward(c_out, c_s)
    want, losses = reference(block, x, stream, c_out, c_s)
    got = dict(norm=block.grads["norm"], x=dx, **{n: block.grads["d" + n] for n in block.weights})
    for n, v in want.items():
        diff = (got[n].cpu().to(D) - v).norm() / v.norm()
        assert diff <= 4 * 2.0 ** -8, (n, float(diff))
    assert ((loss.cpu().to(D) - losses).abs() <= 1e-4 * losses + 1e-30).all()
    # clipping: the norm of all weights' gradients, and the step
    grads = [block.grads["norm"]] + [block.grads["d" + n] for n in block.weights]
    total = sum(float(v.to(D).square().sum()) for v in grads) ** 0.5
    before = [v.clone() for v in grads]
    norm = block.update(0.1, total / 3)
    assert abs(float(norm) / total - 1) <= 1e-6
    for v, b in zip(grads, before):
        assert torch.allclose(v, b / 3, rtol=1e-6, atol=0)
    assert ops.read_error_flags(block.layer.flags) == 0


def test_runs(capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["training_step.py", "--tokens", "256", "--steps", "2"])
    example.main()
    assert capsys.readouterr().out.count("gradients' norm") == 2


def test_low_precision_forward():
    """The norm's 8-bit rows through the shared expert's 8-bit matrices, and its
    bf16 rows through MXFP4 gate matrices: each against the values that the
    codes stand for."""
    T, d, F = 150, 320, 96
    gen = torch.Generator(device="cuda").manual_seed(9)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, res = rand(T, d).bfloat16(), rand(T, d).bfloat16()
    s, y, codes, scales = ops.add_rms_norm(x, torch.ones(d, device="cuda"), residual=res, fp8=True)
    w = {n: rand(1, *shape) / d ** 0.5 for n, shape in dict(gate=(F, d), up=(F, d),
                                                            down=(d, F)).items()}
    q = {n: ops.quantize_weights_fp8_block(v) for n, v in w.items()}
    one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    h8, hs, out = ops.expert_ffn_fp8_block(codes, scales, one, q["gate"], q["up"], q["down"])
    rows = lambda c, sc: (c.cpu().view(torch.float8_e4m3fn).to(D) *  # noqa: E731
                          sc.cpu().to(D).repeat_interleave(128, 1)[:, :c.shape[1]])

    def matrix(n):
        c, sc = q[n][0][0].cpu().view(torch.float8_e4m3fn).to(D), q[n][1][0].cpu().to(D)
        sc = sc.repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]]
        return c * sc
    want = rows(h8, hs) @ matrix("down").t()
    assert (out.cpu().to(D) - want).norm() <= 1e-5 * want.norm()
    a = rows(codes, scales)
    g, u = a @ matrix("gate").t(), a @ matrix("up").t()
    h = g.clamp(-10, 10) * torch.sigmoid(g.clamp(-10, 10)) * u.clamp(-10, 10)
    assert (rows(h8, hs) - h).norm() <= 2.0 ** -4 * h.norm()
    # E4M3 (2^-4) against the bf16 rows
    assert (a - y.cpu().to(D)).norm() <= 2.0 ** -4 * y.cpu().to(D).norm()

    w4, s4 = ops.quantize_mxfp4(rand(2, F, d).bfloat16())
    a4, sa = ops.quantize_mxfp4(y)
    off = torch.tensor([0, 40, T], dtype=torch.int32, device="cuda")
    got = ops.grouped_gemm_mxfp4(a4, sa, off, w4, s4, out_dtype=ops.OUT_F32).cpu().to(D)
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=D)

    def of(c, sc):
        c, sc = c.cpu(), sc.cpu()
        c = torch.stack((c & 15, c >> 4), -1).view(*c.shape[:-1], -1)
        return v[c.long()] * torch.exp2(sc.to(D) - 127).repeat_interleave(32, -1)
    a, m = of(a4, sa), of(w4, s4)
    want = torch.cat([a[:40] @ m[0].t(), a[40:] @ m[1].t()])
    mag = torch.cat([a[:40].abs() @ m[0].abs().t(), a[40:].abs() @ m[1].abs().t()])
    assert ((got - want).abs() <= d * 2.0 ** -24 * mag).all()


def test_flags_of_earlier_steps():
    """What a step's kernels flagged is still there behind the weight update,
    which makes a new layer."""
    w = workloads.small(64, 128, 64, 2, 64, 3, scale=2.5, F_shared=64)
    block = example.Block(w, workloads.make_inputs(w, "cuda"),
                          torch.tensor([0, w.T], dtype=torch.int32, device="cuda"))
    for v in block.grads.values():
        v.zero_()
    block.layer.flags.fill_(ops.FLAG_BAD_EXPERT_ID)
    block.update(0.1, 1.0)
    assert ops.read_error_flags(block.layer.flags) == ops.FLAG_BAD_EXPERT_ID
