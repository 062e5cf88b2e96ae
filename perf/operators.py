"""Measured cases of the layer's 8-bit operators and of its few-token forward.

Four operators, each in a plain form (elementary torch operations) and, with
``own`` set, as the calls that a user makes of this package:

quantise   bf16 or fp32 rows (activations, gradients) or bf16 matrices
           (weights) to E4M3 codes with one power-of-two scale for each block
           of 128 values of a row, or of 128 x 128 values of a matrix:
             X = the least integer with max|v| <= 448 * 2^X, scale = 2^X,
             code = E4M3(v / 2^X), nearest, ties to even.
gemm       out[r, n] = sum_b a_scale[r, b] w_scale[g, n / 128, b]
                       sum_{k in block b} a[r, k] w[g, n, k]
           for the rows r of group g; the forward's products and, on the
           transposed weights, the input gradients.
ffn        the experts' SwiGLU chain on such rows and weights: gate and up
           products, clamp, silu(G) U, quantisation of h along F, down product.
few        the whole layer (router, top-k or hash routing, routed and shared
           experts, combine) for a few tokens, weights in bf16 or in 8 bits
           with a scale for each 128 x 128 block, activations in bf16.
"""
import math

import numpy as np
import torch

own = False

B = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the rows of one decode batch, before the experts' products
        dict(name="quantise-decode", op="quantise", what="rows", dtype="bf16", rows=64, K=4096),
        # the output gradient of a training step (fp32, odd row count, short last block)
        dict(name="quantise-gradient", op="quantise", what="rows", dtype="f32", rows=8191, K=2000),
        # one layer's gate matrices after a weight update
        dict(name="quantise-weights", op="quantise", what="matrix", G=64, N=1024, K=2048),
        # gate product of the 64-expert layer at 4096 tokens, popular and rare experts
        dict(name="gemm-skewed", op="gemm", G=64, rows=24576, K=2048, N=1024, skew=0.8,
             out="bf16"),
        # input gradient of the down projection, 384 experts at 8192 tokens
        dict(name="gemm-input-gradient", op="gemm", G=384, rows=49152, K=4096, N=2048, skew=0.0,
             out="f32"),
        # one dense product, ragged in every direction
        dict(name="gemm-dense-odd", op="gemm", G=1, rows=8191, K=4080, N=2032, skew=0.0,
             out="bf16"),
        # a decode batch of 32 tokens through the 64-expert layer's experts
        dict(name="ffn-decode", op="ffn", G=64, rows=192, d=2048, F=1024, skew=0.5, clamp=10.0),
        # the 384-expert layer's routed experts at 8192 tokens
        dict(name="ffn-prefill", op="ffn", G=384, rows=49152, d=4096, F=2048, skew=0.0,
             clamp=10.0),
        # one token of one sequence through the 64-expert layer: latency
        dict(name="few-1-bf16", op="few", T=1, E=64, k=6, d=2048, F=1024, Fs=1024, w="bf16",
             mode="topk", n_bias=1, clamp=10.0, scale=1.0),
        # one token through the 384-expert layer, 8-bit weights
        dict(name="few-1-fp8", op="few", T=1, E=384, k=6, d=4096, F=2048, Fs=2048, w="fp8",
             mode="topk", n_bias=2, clamp=10.0, scale=2.5),
        # a small serving batch through the 384-expert layer, bf16 weights
        dict(name="few-8-bf16", op="few", T=8, E=384, k=6, d=4096, F=2048, Fs=2048, w="bf16",
             mode="topk", n_bias=1, clamp=10.0, scale=2.5),
        # a larger batch, hash routed, 8-bit weights, odd count
        dict(name="few-33-fp8-hash", op="few", T=33, E=384, k=6, d=4096, F=2048, Fs=2048,
             w="fp8", mode="hash", n_bias=0, clamp=10.0, scale=2.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, hi):
    """A row count: odd, so that the last tile is a ragged one."""
    return _log(rng, 1, hi) | 1


def _width(rng, lo, hi, m):
    """A matrix side: a power of two, or an odd multiple of m."""
    n = _log(rng, lo, hi)
    return 1 << (n.bit_length() - 1) if rng.random() < 0.5 else n // (2 * m) * 2 * m + m


def draw(rng):
    op = rng.choice(["quantise", "gemm", "ffn", "few", "gemm", "few"])
    if op == "quantise":
        if rng.random() < 0.7:
            return dict(op=op, what="rows", dtype=rng.choice(["bf16", "f32"]),
                        rows=_odd(rng, 49151), K=_width(rng, 64, 4096, 16))
        return dict(op=op, what="matrix", G=_log(rng, 1, 64), N=_width(rng, 64, 2048, 16),
                    K=_width(rng, 64, 4096, 16))
    if op in ("gemm", "ffn"):
        G = 1 if rng.random() < 0.2 else _log(rng, 2, 384)
        rows = _odd(rng, 49151)
        a, b = _width(rng, 64, 4096, 16), _width(rng, 64, 2048, 16)
        skew = rng.choice([0.0, 0.5, 0.8])
        if G > 64:
            skew = min(skew, 0.5)
        if op == "ffn":
            return dict(op=op, G=G, rows=rows, d=a, F=b, skew=skew,
                        clamp=rng.choice([1.0, 10.0, 1e30]))
        if rng.random() < 0.5:
            a, b = b, a
        return dict(op=op, G=G, rows=rows, K=a, N=b, skew=skew, out=rng.choice(["bf16", "f32"]))
    E = _log(rng, 8, 384)
    mode = rng.choice(["topk", "topk", "hash"])
    F = _width(rng, 64, 2048, 64)
    return dict(op=op, T=_log(rng, 1, 33), E=E, k=rng.randint(1, min(8, E) if E < 200 else 6),
                d=_width(rng, 128, 4096, 64), F=F, Fs=rng.choice([0, F, 64]),
                w=rng.choice(["bf16", "fp8"]), mode=mode,
                n_bias=0 if mode == "hash" else rng.choice([0, 1, 2]),
                clamp=rng.choice([1.0, 10.0]), scale=rng.choice([1.0, 2.5]))


# ----------------------------------------------------------------- inputs --
DEV = "cuda"


def _nb(n):
    return -(-n // B)


def _codes(shape, gen):
    """E4M3 codes of normal weights: the block maximum near the format's, as a
    quantiser leaves them, the values from its normals down to its zeros."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        v = torch.randn(n, generator=gen, device=DEV, dtype=torch.float16)
        flat[i:i + n] = v.mul_(90.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _weights8(G, N, K, gen):
    """8-bit matrices of standard deviation near 1 / sqrt(K), the blocks'
    scales any fp32 values, as checkpoints hold them."""
    s = torch.rand((G, _nb(N), _nb(K)), generator=gen, device=DEV) * 0.5 + 0.75
    return _codes((G, N, K), gen), s / (90.0 * math.sqrt(K))


def _weights16(shape, gen):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        v = torch.randn(n, generator=gen, device=DEV, dtype=torch.bfloat16)
        flat[i:i + n] = v.mul_(1.0 / math.sqrt(shape[-1]))
    return out


def _groups(case, seed):
    """Row offsets of the groups: popularity of rank r as r^-skew, ranks
    permuted; groups without rows occur."""
    rng = np.random.default_rng(seed)
    G, rows = case["G"], case["rows"]
    p = (rng.permutation(G) + 1.0) ** -case["skew"]
    counts = rng.multinomial(rows, p / p.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), int(counts.max())


def _rows8(rows, K, gen):
    """Quantised rows: normal values under per-row magnitudes that vary."""
    a = torch.randn((rows, K), generator=gen, device=DEV)
    a *= torch.rand((rows, 1), generator=gen, device=DEV) * 3 + 0.1
    return _quantise_rows(a)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    st = dict(case=case)
    op = case["op"]
    if op == "quantise":
        shape = ((case["rows"], case["K"]) if case["what"] == "rows"
                 else (case["G"], case["N"], case["K"]))
        a = torch.randn(shape, generator=gen, device=DEV)
        # channels of different magnitude, as activations and gradients have
        a *= torch.exp2(torch.randn((case["K"],), generator=gen, device=DEV) * 2)
        st["a"] = a if case.get("dtype") == "f32" else a.to(torch.bfloat16)
        return st
    if op in ("gemm", "ffn"):
        offs, st["cap"] = _groups(case, seed)
        st["offsets"] = torch.from_numpy(offs).to(DEV)
        G = case["G"]
        if op == "gemm":
            st["a"], st["as"] = _rows8(case["rows"], case["K"], gen)
            st["w"], st["ws"] = _weights8(G, case["N"], case["K"], gen)
        else:
            d, F = case["d"], case["F"]
            st["a"], st["as"] = _rows8(case["rows"], d, gen)
            for n, (o, i) in dict(gate=(F, d), up=(F, d), down=(d, F)).items():
                st["w_" + n], st["w_" + n + "_scale"] = _weights8(G, o, i, gen)
        return st
    T, E, k, d, F, Fs = (case[n] for n in ("T", "E", "k", "d", "F", "Fs"))
    st["x"] = torch.randn((T, d), generator=gen, device=DEV).to(torch.bfloat16)
    w = dict(w_g=_weights16((E, d), gen))
    for n, shape in dict(w_gate=(E, F, d), w_up=(E, F, d), w_down=(E, d, F), s_gate=(Fs, d),
                         s_up=(Fs, d), s_down=(d, Fs)).items():
        if n[0] == "s" and Fs == 0:
            continue
        if case["w"] == "bf16":
            w[n] = _weights16(shape, gen)
        else:
            c, s = _weights8(shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], gen)
            w[n], w[n + "_scale"] = c.view(shape), s if len(shape) == 3 else s[0]
    st["modality"] = st["input_ids"] = None
    if case["mode"] == "hash":
        V = 4096
        w["tid2eid"] = torch.rand((V, E), generator=gen, device=DEV).argsort(1)[:, :k].to(
            torch.int32).contiguous()
        st["input_ids"] = torch.randint(0, V, (T,), generator=gen, device=DEV,
                                        dtype=torch.int32)
    elif case["n_bias"]:
        w["score_bias"] = torch.rand((case["n_bias"], E), generator=gen, device=DEV) * 0.2 - 0.1
        if case["n_bias"] == 2:
            st["modality"] = (torch.rand((T,), generator=gen, device=DEV) < 0.3).to(torch.uint8)
    st["weights"] = w
    if own:  # the handle that a serving program keeps: weights, sizes, workspace
        from sparse_moe_layer_04_amd import ops
        st["layer"] = ops.MoeLayer(
            T, d, E, k, F, Fs, w, n_bias=case["n_bias"], V=4096 if case["mode"] == "hash" else 0,
            mode=ops.MODE_HASH if case["mode"] == "hash" else ops.MODE_TOPK,
            scale=case["scale"], clamp_limit=case["clamp"],
            packed="fp8_block" if case["w"] == "fp8" else False)
    return st


# ------------------------------------------------------------ plain forms --
def _pow2(amax):
    """2^X, X the least integer with amax <= 448 * 2^X (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    X = (e - torch.where(m <= 0.875, 9, 8)).clamp(-126, 120) * (amax > 0)
    return ((X + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(v):
    rows, K = v.shape
    return torch.nn.functional.pad(v, (0, _nb(K) * B - K)).view(rows, _nb(K), B)


def _quantise_rows(v):
    K = v.shape[1]
    b = _blocks(v.float())
    s = _pow2(b.abs().amax(-1))
    q = (b / s[..., None]).to(torch.float8_e4m3fn)
    return q.view(v.shape[0], -1)[:, :K].contiguous(), s


def _quantise_matrix(w):
    G, N, K = w.shape
    p = torch.nn.functional.pad(w.float(), (0, _nb(K) * B - K, 0, _nb(N) * B - N))
    p = p.view(G, _nb(N), B, _nb(K), B)
    s = _pow2(p.abs().amax((2, 4)))
    q = (p / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(G, _nb(N) * B, _nb(K) * B)[:, :N, :K].contiguous(), s


def _rows(q, s, dt=torch.float32):
    """The values of quantised rows."""
    return q.to(dt) * s.to(dt).repeat_interleave(B, 1)[:, :q.shape[1]]


def _matrix(q, s, dt=torch.float32):
    """The values of quantised matrices [..., N, K]."""
    N, K = q.shape[-2:]
    s = s.to(dt).repeat_interleave(B, -2)[..., :N, :].repeat_interleave(B, -1)[..., :K]
    return q.to(dt) * s


def _pad_groups(st, v):
    """[G, cap, K]: each group's rows (past its end: rows that nothing reads)."""
    at = st["offsets"][:-1, None].long() + torch.arange(st["cap"], device=v.device)
    return v[at.clamp(max=v.shape[0] - 1)]


def _unpad_groups(st, v, rows):
    r = torch.arange(rows, device=v.device)
    g = torch.searchsorted(st["offsets"][1:].long(), r, right=True)
    return v[g, r - st["offsets"].long()[g]]


def _swiglu(G, U, clamp):
    G, U = G.clamp(-clamp, clamp), U.clamp(-clamp, clamp)
    return G / (1 + torch.exp(-G)) * U


def _plain_gemm(st):
    out = torch.bmm(_pad_groups(st, _rows(st["a"], st["as"])),
                    _matrix(st["w"], st["ws"]).transpose(1, 2))
    out = _unpad_groups(st, out, st["a"].shape[0])
    return out if st["case"]["out"] == "f32" else out.to(torch.bfloat16)


def _plain_ffn(st):
    a = _pad_groups(st, _rows(st["a"], st["as"]))
    G = torch.bmm(a, _matrix(st["w_gate"], st["w_gate_scale"]).transpose(1, 2))
    U = torch.bmm(a, _matrix(st["w_up"], st["w_up_scale"]).transpose(1, 2))
    h = _swiglu(G, U, st["case"]["clamp"])
    q, s = _quantise_rows(h.view(-1, h.shape[-1]))
    h = _rows(q, s).view(h.shape)
    y = torch.bmm(h, _matrix(st["w_down"], st["w_down_scale"]).transpose(1, 2))
    return _unpad_groups(st, y, st["a"].shape[0]).to(torch.bfloat16)


def _route(st, logits):
    """(expert, weight) of each token's k choices; scores in fp32, equal ones
    to the lower index."""
    c, w = st["case"], st["weights"]
    s = torch.sigmoid(logits)
    if c["mode"] == "hash":
        ids = w["tid2eid"][st["input_ids"].long()].long()
    else:
        r = s.float()
        if c["n_bias"]:
            m = st["modality"]
            r = r + w["score_bias"].float()[0 if m is None else m.long()]
        ids = torch.sort(r, dim=1, descending=True, stable=True)[1][:, :c["k"]]
    g = s.gather(1, ids)
    return ids, g / g.sum(1, keepdim=True) * c["scale"]


def _take(w, name, at, dt=torch.float32):
    """The fp32 (64-bit) matrices of the chosen experts, or the shared ones."""
    v = w[name] if at is None else w[name].view(torch.uint8)[at].view(w[name].dtype) \
        if w[name].dtype == torch.float8_e4m3fn else w[name][at]
    if v.dtype == torch.bfloat16:
        return v.to(dt)
    s = w[name + "_scale"]
    return _matrix(v, s if at is None else s[at], dt)


def _plain_few(st):
    c, w = st["case"], st["weights"]
    T, k, d = c["T"], c["k"], c["d"]
    x = st["x"].float()
    # the logits in 64 bits: the choice of experts lies next to a border
    logits = (st["x"].double() @ w["w_g"].double().t()).float()
    ids, wt = _route(st, logits)
    at = ids.reshape(-1)
    xr = x.repeat_interleave(k, 0)[:, :, None]
    h = _swiglu(torch.bmm(_take(w, "w_gate", at), xr), torch.bmm(_take(w, "w_up", at), xr),
                c["clamp"])
    y = torch.bmm(_take(w, "w_down", at), h.to(torch.bfloat16).float())
    y = (y.view(T, k, d) * wt[:, :, None]).sum(1)
    if c["Fs"]:
        h = _swiglu(x @ _take(w, "s_gate", None).t(), x @ _take(w, "s_up", None).t(), c["clamp"])
        y = y + h.to(torch.bfloat16).float() @ _take(w, "s_down", None).t()
    return dict(y=y.to(torch.bfloat16), w=wt)


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "quantise":
            return (_quantise_rows if c["what"] == "rows" else _quantise_matrix)(st["a"])
        return dict(gemm=_plain_gemm, ffn=_plain_ffn, few=_plain_few)[op](st)
    from sparse_moe_layer_04_amd import ops
    if op == "quantise":
        q, s = (ops.quantize_fp8_block if c["what"] == "rows"
                else ops.quantize_weights_fp8_block)(st["a"])
        return q.view(torch.float8_e4m3fn), s
    if op == "gemm":
        return ops.grouped_gemm_fp8_block(
            st["a"], st["as"], st["offsets"], st["w"], st["ws"],
            out_dtype=ops.OUT_F32 if c["out"] == "f32" else ops.OUT_BF16)
    if op == "ffn":
        return ops.expert_ffn_fp8_block(
            st["a"], st["as"], st["offsets"], (st["w_gate"], st["w_gate_scale"]),
            (st["w_up"], st["w_up_scale"]), (st["w_down"], st["w_down_scale"]),
            clamp_limit=c["clamp"], out_dtype=ops.OUT_BF16)[2]
    w = torch.empty((c["T"], c["k"]), dtype=torch.float32, device=st["x"].device)
    y = st["layer"].forward_few(st["x"], input_ids=st["input_ids"], modality=st["modality"], w=w)
    return dict(y=y, w=w)


# ------------------------------------------------------------ exact values --
def _e4m3(v):
    """The nearest E4M3 value of v (|v| <= 448), ties to even, in 64 bits."""
    e = torch.frexp(v)[1] - 1                     # floor(log2 |v|)
    step = _two_to(e.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _two_to(X):
    """2^X in 64 bits, exactly: the exponent's bits."""
    return ((X.long() + 1023) << 52).view(torch.float64)


def _scale64(amax):
    X = torch.floor(torch.log2(amax.clamp(min=1e-300))).long() - 10  # (too small)
    for _ in range(3):
        X = torch.where(E4M3_MAX * _two_to(X) < amax, X + 1, X)
    return torch.where(amax > 0, _two_to(X.clamp(-126, 120)), torch.ones_like(amax))


def _exact_rows(v):
    """(codes' values, scales) of rows in 64 bits."""
    q, s = torch.empty_like(v), torch.empty(v.shape[0], _nb(v.shape[1]), dtype=v.dtype,
                                            device=v.device)
    for b in range(_nb(v.shape[1])):
        p = v[:, b * B:(b + 1) * B]
        s[:, b] = _scale64(p.abs().amax(1))
        q[:, b * B:(b + 1) * B] = _e4m3(p / s[:, b:b + 1])
    return q, s


def exact(case, seed):
    D = torch.float64
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        if case["what"] == "rows":
            return _exact_rows(st["a"].to(D))
        q = torch.empty(st["a"].shape, dtype=D, device=DEV)
        s = torch.empty((case["G"], _nb(case["N"]), _nb(case["K"])), dtype=D, device=DEV)
        for n in range(s.shape[1]):
            for b in range(s.shape[2]):
                p = st["a"][:, n * B:(n + 1) * B, b * B:(b + 1) * B].to(D)
                s[:, n, b] = _scale64(p.abs().amax((1, 2)))
                q[:, n * B:(n + 1) * B, b * B:(b + 1) * B] = _e4m3(p / s[:, n, b, None, None])
        return q, s
    if op in ("gemm", "ffn"):
        offs = st["offsets"].tolist()
        y = torch.empty((case["rows"], case["N"] if op == "gemm" else case["d"]), dtype=D,
                        device=DEV)
        for g in range(case["G"]):
            lo, hi = offs[g], offs[g + 1]
            if lo == hi:
                continue
            a = _rows(st["a"][lo:hi], st["as"][lo:hi], D)
            if op == "gemm":
                y[lo:hi] = a @ _matrix(st["w"][g], st["ws"][g], D).t()
                continue
            wg, wu, wd = (_matrix(st[n][g], st[n + "_scale"][g], D)
                          for n in ("w_gate", "w_up", "w_down"))
            q, s = _exact_rows(_swiglu(a @ wg.t(), a @ wu.t(), case["clamp"]))
            y[lo:hi] = (q * s.repeat_interleave(B, 1)[:, :q.shape[1]]) @ wd.t()
        return y
    w, x = st["weights"], st["x"].to(D)
    ids, wt = _route(st, x @ w["w_g"].to(D).t())
    y = torch.zeros_like(x)
    for t in range(case["T"]):
        for j in range(case["k"]):
            e = ids[t, j]
            m = [w[n][e].to(D) if case["w"] == "bf16"
                 else _matrix(w[n][e], w[n + "_scale"][e], D)
                 for n in ("w_gate", "w_up", "w_down")]
            h = _swiglu(m[0] @ x[t], m[1] @ x[t], case["clamp"])
            y[t] += wt[t, j] * (m[2] @ h.to(torch.bfloat16).to(D))
    if case["Fs"]:
        m = [_take(w, n, None, D) for n in ("s_gate", "s_up", "s_down")]
        h = _swiglu(x @ m[0].t(), x @ m[1].t(), case["clamp"])
        y += h.to(torch.bfloat16).to(D) @ m[2].t()
    return dict(y=y, w=wt)


# ------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "quantise":
        if case["what"] == "rows":
            n, blocks = case["rows"] * case["K"], case["rows"] * _nb(case["K"])
        else:
            n = case["G"] * case["N"] * case["K"]
            blocks = case["G"] * _nb(case["N"]) * _nb(case["K"])
        return dict(bytes=n * ((4 if case.get("dtype") == "f32" else 2) + 1) + 4 * blocks,
                    flops=2 * n)
    if op in ("gemm", "ffn"):
        G, rows = case["G"], case["rows"]
        used = G * (1 - (1 - 1 / G) ** rows) if G > 1 else 1  # groups with rows
        i, o = (case["K"], case["N"]) if op == "gemm" else (case["d"], case["d"])
        per = i * o if op == "gemm" else 3 * case["d"] * case["F"]
        out = 4 if case.get("out") == "f32" else 2
        return dict(bytes=used * per * (1 + 4 / B / B) + rows * (i * (1 + 4 / B) + o * out),
                    flops=2 * rows * per)
    T, E, k, d, F, Fs = (case[n] for n in ("T", "E", "k", "d", "F", "Fs"))
    used = E * (1 - (1 - k / E) ** T)
    size = 2 if case["w"] == "bf16" else 1 + 4 / B / B
    return dict(bytes=3 * d * (used * F + Fs) * size + E * d * 2 + T * d * 4,
                flops=2 * T * d * (3 * (k * F + Fs) + E))
