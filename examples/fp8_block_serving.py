"""One MoE layer served on 8-bit weights with block scales: a prompt through
the pieces of the layer, then single tokens through one call each.

    python examples/fp8_block_serving.py [--config 1] [--prompt 2048] [--steps 64]

The weights are quantised once, to E4M3 codes with one scale for each
128 x 128 block (a checkpoint in that format is loaded as it is), and both
phases read the same arrays:

* prefill: router and routes, permutation, the rows quantised (one scale for
  each 128 of a row), the grouped expert FFN on the 8-bit rows, the shared
  expert as a group of its own, the weighted combine;
* decode: ``MoeLayer.forward_few`` on up to FEW_MAX_T tokens with bf16
  activations, captured once into a HIP graph and replayed for every step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_moe_layer_04_amd import ops, workloads  # noqa: E402

MATRICES = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")


def quantized_layer(w, inputs, tokens=ops.FEW_MAX_T, out_dtype=ops.OUT_BF16):
    """The MoeLayer of workload w on 8-bit copies of its bf16 matrices."""
    weights = dict(inputs)
    for n in MATRICES:
        if weights.get(n) is not None:
            weights[n], weights[n + "_scale"] = ops.quantize_weights_fp8_block(weights[n])
    n_bias = 0 if inputs.get("score_bias") is None else inputs["score_bias"].shape[0]
    return ops.MoeLayer(tokens, w.d, w.E, w.k, w.F, w.Fs, weights, mode=w.mode, n_bias=n_bias,
                        V=w.V, scale=w.scale, clamp_limit=w.clamp_limit,
                        clamp_mode=w.clamp_mode, out_dtype=out_dtype, packed="fp8_block")


def prefill(layer, x, input_ids=None, modality=None):
    """The layer on any number of tokens x [T, d] bf16: returns (y, ids)."""
    c, w = layer.cfg, layer.weights
    ffn = dict(clamp_limit=c.clamp_limit, clamp_mode=c.clamp_mode, out_dtype=ops.OUT_F32)
    logits = ops.gate_logits(x, w["w_g"], w.get("logit_offset"))
    ids, topk_w = ops.route(logits, c.k, c.scale, w.get("score_bias"), modality, input_ids,
                            w.get("tid2eid"), c.mode, layer.flags)
    p = ops.permute(ids, x, c.E, layer.flags)
    pair = lambda n: (w[n], w[n + "_scale"])  # noqa: E731
    y_perm = ops.expert_ffn_fp8_block(*ops.quantize_fp8_block(p["x_perm"]), p["offsets"],
                                      pair("w_gate"), pair("w_up"), pair("w_down"), **ffn)[2]
    y_shared = None
    if c.F_shared > 0:
        one = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
        group = lambda n: (w[n][None], w[n + "_scale"][None])  # noqa: E731
        y_shared = ops.expert_ffn_fp8_block(*ops.quantize_fp8_block(x), one, group("s_gate"),
                                            group("s_up"), group("s_down"), **ffn)[2]
    return ops.combine(y_perm, p["dest"], topk_w, y_shared, c.out_dtype), ids


class Decoder:
    """forward_few on a fixed number of tokens, captured into a HIP graph, with
    a workspace of its own (decoders of one layer may run at once)."""

    def __init__(self, layer, tokens=1, input_ids=None, modality=None):
        dt = torch.float32 if layer.cfg.out_dtype == ops.OUT_F32 else torch.bfloat16
        self.x = torch.zeros((tokens, layer.cfg.d), dtype=torch.bfloat16, device=layer.device)
        self.y = torch.empty((tokens, layer.cfg.d), dtype=dt, device=layer.device)
        self.ids = torch.empty((tokens, layer.cfg.k), dtype=torch.int32, device=layer.device)
        self.ws = layer.few_workspace()
        run = lambda: layer.forward_few(self.x, input_ids, modality, y=self.y,  # noqa: E731
                                        ids=self.ids, ws=self.ws)
        stream = torch.cuda.Stream(layer.device)
        stream.wait_stream(torch.cuda.current_stream(layer.device))
        with torch.cuda.stream(stream):
            run()                                  # (kernels loaded)
        torch.cuda.current_stream(layer.device).wait_stream(stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            run()

    def step(self, x):
        """y and ids of the tokens x; both are overwritten by the next step."""
        self.x.copy_(x)
        self.graph.replay()
        return self.y, self.ids


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--config", type=int, default=1, choices=(0, 1, 2),
                    help="workload: 64 experts (1), 384 experts (2), a tiny one (0)")
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    w = workloads.WORKLOADS[args.config]
    dev = torch.device("cuda")
    layer = quantized_layer(w, workloads.make_inputs(w, dev))
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn((args.prompt + args.steps, w.d), generator=g, device=dev).bfloat16()

    prefill(layer, x[:args.prompt])                # (kernels loaded, memory cached)
    decoder = Decoder(layer)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    prefill(layer, x[:args.prompt])
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    for t in range(args.steps):
        decoder.step(x[args.prompt + t:args.prompt + t + 1])
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    if ops.read_error_flags(layer.flags):
        raise ops.MoeError("the layer raised its error flags")
    print(f"{w.name}: prefill of {args.prompt} tokens {(t1 - t0) * 1e3:.2f} ms, "
          f"decode {(t2 - t1) / max(args.steps, 1) * 1e6:.1f} us a token")
    last = x[-1:]
    a = prefill(layer, last)[0].double()
    b = decoder.step(last)[0].double()
    print(f"prefill (8-bit rows) against decode (bf16 rows), one token: relative difference "
          f"{float((a - b).norm() / b.norm()):.3f}")


if __name__ == "__main__":
    main()
