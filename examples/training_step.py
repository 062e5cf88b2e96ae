"""Training steps of one block: norm with the residual's addition, the MoE
layer, the balance loss of its routes, the way back, clipping, SGD.

    python examples/training_step.py [--tokens 1024] [--steps 5]

* forward: ``add_rms_norm`` adds the last block's output to the residual stream
  and normalises it, the layer runs on the result, ``balance_loss`` counts the
  tokens of each expert (text and image tokens apart, where there are both);
* backward: the layer's gradients and the balance loss's gradient in the router's logits,
  taken through the router's matrix by the grouped products, then
  ``rms_norm_backward``, whose result is the gradient of the block's input and
  of the stream;
* the gradients of all weights lie in buffers that are kept, so one ``GradClip``
  clips them in every step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_moe_layer_04_amd import ops, workloads  # noqa: E402

MATRICES = ("w_g", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")


class Block:
    """Workload w's layer behind a norm; the number of experts is a multiple of
    64 (the router's input gradient is a grouped product over them)."""

    def __init__(self, w, inputs, offsets, eps=1e-6, balance=0.01):
        self.w, self.inputs, self.offsets, self.eps = w, dict(inputs), offsets, eps
        dev = inputs["x"].device
        self.norm = torch.ones(w.d, device=dev)
        self.modality = inputs["modality"] if w.n_bias == 2 else None
        classes = 1 if self.modality is None else 2
        groups = (offsets.numel() - 1) * classes
        self.d_loss = torch.full((offsets.numel() - 1, classes), balance / groups, device=dev)
        self.all_tokens = torch.tensor([0, w.T], dtype=torch.int32, device=dev)
        like = lambda n: torch.empty(self.inputs[n].shape, device=dev)  # noqa: E731
        self.weights = [n for n in MATRICES if self.inputs.get(n) is not None]
        self.grads = dict(dx=torch.empty((w.T, w.d), device=dev),
                          norm=torch.empty(w.d, device=dev),
                          **{"d" + n: like(n) for n in self.weights})
        self.flags = torch.zeros(1, dtype=torch.int32, device=dev)     # of all steps
        self.clip = ops.GradClip([self.grads["norm"]] + [self.grads["d" + n] for n in self.weights])
        self.load()

    def load(self):
        """The layouts of the layer's kernels, after a weight update."""
        self.layer = ops.MoeLayer.from_workload(self.w, self.inputs, out_dtype=ops.OUT_F32,
                                                packed=True)
        self.layer.flags = self.flags
        self.w_g_t = ops.pack_weights(self.inputs["w_g"].t().contiguous(), 256)

    def forward(self, x, stream):
        """x [T, d], the last block's output, and the residual stream: returns
        this block's output (fp32), the stream behind the addition, and the
        balance losses."""
        w, dev = self.w, x.device
        self.s, self.y, _, _ = ops.add_rms_norm(x, self.norm, residual=stream, eps=self.eps)
        self.logits = torch.empty((w.T, w.E), device=dev)
        self.ids = torch.empty((w.T, w.k), dtype=torch.int32, device=dev)
        out = self.layer.forward(self.y, modality=self.modality, logits=self.logits, ids=self.ids)
        loss, self.counts = ops.balance_loss(self.logits, self.ids, self.offsets, self.modality,
                                             flags=self.flags)
        return out, self.s, loss

    def backward(self, d_out, d_stream=None):
        """Gradients for those of the output (fp32) and of the stream (None:
        zero), the balance losses' with their weight: fills self.grads and
        returns the gradient of x and of the stream in front."""
        g = self.grads
        self.layer.backward(self.y, d_out, modality=self.modality,
                            grads={n: v for n, v in g.items() if n != "norm"})
        d_logits = ops.balance_loss_backward(self.logits, self.ids, self.counts, self.d_loss,
                                             self.offsets, self.modality).bfloat16()
        g["dx"] += ops.grouped_gemm_packed(d_logits, self.all_tokens, self.w_g_t, 1, self.w.d)
        g["dw_g"] += ops.grouped_wgrad(d_logits, self.y, None)[0]
        return ops.rms_norm_backward(self.s, self.norm, g["dx"], eps=self.eps, d_res=d_stream,
                                     dw=g["norm"])[0]

    def update(self, rate, max_norm):
        """Clips the gradients, takes an SGD step, returns their norm before."""
        norm = self.clip.clip(max_norm)
        self.norm -= rate * self.grads["norm"]
        for n in self.weights:
            self.inputs[n] = (self.inputs[n].float() - rate * self.grads["d" + n]).bfloat16()
        self.load()
        return norm


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=5)
    args = ap.parse_args()
    w = workloads.small(args.tokens, 512, 64, 6, 256, 3, scale=2.5, F_shared=256)
    dev = torch.device("cuda")
    inputs = workloads.make_inputs(w, dev)
    half = torch.tensor([0, w.T // 2, w.T], dtype=torch.int32, device=dev)
    block = Block(w, inputs, half)
    target = torch.randn((w.T, w.d), device=dev)
    stream = torch.zeros((w.T, w.d), dtype=torch.bfloat16, device=dev)
    for step in range(args.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        out, s, balance = block.forward(inputs["x"], stream)
        error = out + s.float() - target
        block.backward(error / w.T, error / w.T)
        norm = block.update(0.1, 1.0)
        torch.cuda.synchronize()
        print(f"step {step}: error {float(error.square().mean()):.4f}, balance "
              f"{float(balance.mean()):.4f}, gradients' norm {float(norm):.3f}, "
              f"{(time.perf_counter() - t) * 1e3:.1f} ms")
    if ops.read_error_flags(block.flags):
        raise ops.MoeError("a step raised the error flags")


if __name__ == "__main__":
    main()
