"""The layer forward for a few tokens against a plain 64-bit implementation.

Logits: fp32 sums of d exact bf16 products, within 2 d 2^-24 sum |terms| of
the 64-bit ones.  Routes and weights: bit for bit those of moe_route on the
logits that the call returns.  y: from those routes in 64 bits with h rounded
to bf16 as the layer does; the kernel's h is that or, where the fp32 sum lies
next to a rounding border, a neighbour (one step, 2^-7 of one of F terms), so
an fp32 y is within 1e-2 of the output's RMS everywhere and within 1e-3 in
the 2-norm; a bf16 y adds its rounding, 2^-8 of the value.
"""
import pytest
import torch

from sparse_moe_layer_04_amd import ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
D = torch.float64
MATS = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make(T, d, E, k, F, Fs, fp8, seed, mode=ops.MODE_TOPK, n_bias=0, V=50, out=ops.OUT_F32,
         clamp=10.0, clamp_mode=0, scale=2.5, offset=False):
    g = gen(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    w = dict(w_g=(rnd(E, d) / d ** 0.5).bfloat16())
    shapes = dict(w_gate=(E, F, d), w_up=(E, F, d), w_down=(E, d, F))
    if Fs:
        shapes.update(s_gate=(Fs, d), s_up=(Fs, d), s_down=(d, Fs))
    for n, s in shapes.items():
        v = rnd(*s) / s[-1] ** 0.5
        if fp8:
            w[n], w[n + "_scale"] = ops.quantize_weights_fp8_block(v)
            w[n + "_scale"] *= torch.rand(w[n + "_scale"].shape, generator=g, device=DEV) + 0.5
        else:
            w[n] = v.bfloat16()
    if offset:
        w["logit_offset"] = rnd(E)
    if n_bias:
        w["score_bias"] = rnd(n_bias, E) * 0.2
    if mode == ops.MODE_HASH:
        w["tid2eid"] = rnd(V, E).argsort(1)[:, :k].to(torch.int32).contiguous()
    layer = ops.MoeLayer(T, d, E, k, F, Fs, w, mode=mode, n_bias=n_bias,
                         V=V if mode == ops.MODE_HASH else 0, scale=scale, clamp_limit=clamp,
                         clamp_mode=clamp_mode, out_dtype=out,
                         packed="fp8_block" if fp8 else False)
    x = rnd(T, d).bfloat16()
    ids = mod = None
    if mode == ops.MODE_HASH:
        ids = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    elif n_bias == 2:
        mod = (torch.rand((T,), generator=g, device=DEV) < 0.5).to(torch.uint8)
    return layer, w, x, ids, mod


def matrix(w, n, e=None):
    c = w[n] if e is None else w[n][e]
    if c.dtype == torch.bfloat16:
        return c.to(D)
    s = w[n + "_scale"] if e is None else w[n + "_scale"][e]
    s = s.to(D).repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]]
    return c.view(torch.float8_e4m3fn).to(D) * s


def ffn(layer, w, names, e, x):
    c = layer.cfg
    g, u = x @ matrix(w, names[0], e).t(), x @ matrix(w, names[1], e).t()
    L = c.clamp_limit
    g = g.clamp(-L, L) if c.clamp_mode == 0 else g.clamp(max=L)
    h = g / (1 + torch.exp(-g)) * u.clamp(-L, L)
    return h.to(torch.bfloat16).to(D) @ matrix(w, names[2], e).t()


def plain(layer, w, x, ids, wt):
    x = x.to(D)
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e >= 0:
                y[t] += wt[t, j].to(D) * ffn(layer, w, MATS[:3], e, x[t])
    if layer.cfg.F_shared:
        y += ffn(layer, w, MATS[3:], None, x)
    return y


def check(layer, w, x, in_ids, mod):
    c = layer.cfg
    T = x.shape[0]
    logits = torch.full((T, c.E), 9.0, device=DEV)
    ids = torch.full((T, c.k), -7, dtype=torch.int32, device=DEV)
    wt = torch.full((T, c.k), 9.0, device=DEV)
    y = layer.forward_few(x, input_ids=in_ids, modality=mod, logits=logits, ids=ids, w=wt)
    ref = x.to(D) @ w["w_g"].to(D).t()
    mag = x.to(D).abs() @ w["w_g"].to(D).abs().t()
    if "logit_offset" in w:
        ref, mag = ref + w["logit_offset"].to(D), mag + w["logit_offset"].to(D).abs()
    assert bool(((logits.to(D) - ref).abs() <= 2 * (c.d + 1) * 2.0 ** -24 * mag).all())
    rid, rw = ops.route(logits, c.k, c.scale, score_bias=w.get("score_bias"), modality=mod,
                        input_ids=in_ids, tid2eid=w.get("tid2eid"), mode=c.mode)
    assert torch.equal(ids, rid)
    assert torch.equal(wt, rw)
    ref = plain(layer, w, x, ids, wt)
    err = (y.to(D) - ref).abs()
    rms = float(ref.pow(2).mean().sqrt())
    bf16 = c.out_dtype == ops.OUT_BF16
    bound = 1e-2 * rms + (2.0 ** -8 * ref.abs() if bf16 else 0)
    assert bool((err <= bound).all()), float(err.max()) / rms
    assert float(err.norm()) <= (3.5e-3 if bf16 else 1e-3) * float(ref.norm())
    # without the optional outputs, and again: the same bits
    assert torch.equal(layer.forward_few(x, input_ids=in_ids, modality=mod), y)
    return y


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,F,Fs", [
    (1, 64, 8, 2, 64, 0), (1, 128, 8, 8, 64, 64), (2, 192, 17, 3, 320, 64),
    (7, 256, 64, 6, 192, 256), (16, 320, 33, 4, 64, 128), (17, 128, 9, 8, 448, 64),
    (33, 576, 100, 6, 128, 64), (64, 256, 8, 8, 128, 128), (64, 128, 1, 1, 64, 64),
    (5, 2048, 64, 6, 1024, 1024), (1, 4096, 384, 6, 2048, 2048), (3, 128, 1024, 8, 64, 0)])
def test_topk(T, d, E, k, F, Fs, fp8):
    check(*make(T, d, E, k, F, Fs, fp8, T + d + E))


# router and shared expert in more workgroups than 256 CUs hold at once, in as
# many, and a last router strip of few experts
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,F,Fs", [
    (1, 64, 240, 2, 64, 2048), (1, 1216, 384, 6, 64, 2048), (16, 128, 511, 3, 64, 2048),
    (33, 192, 1000, 2, 64, 2048), (64, 64, 1024, 8, 64, 1984), (17, 128, 17, 2, 64, 2048),
    (64, 128, 200, 2, 64, 2112)])
def test_router_beside_the_shared_expert(T, d, E, k, F, Fs, fp8):
    check(*make(T, d, E, k, F, Fs, fp8, T + d + E))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(n_bias=1), dict(n_bias=2), dict(n_bias=2, offset=True), dict(mode=ops.MODE_HASH),
    dict(clamp=0.5), dict(clamp=0.5, clamp_mode=1), dict(clamp=float("inf")),
    dict(out=ops.OUT_BF16), dict(scale=0.0)])
def test_modes(kw, fp8):
    check(*make(9, 256, 24, 4, 192, 128, fp8, 5, **kw))


@pytest.mark.parametrize("fp8", [False, True])
def test_fewer_tokens_than_the_layer(fp8):
    layer, w, x, _, _ = make(40, 256, 24, 4, 192, 128, fp8, 6)
    whole = layer.forward_few(x)
    for t in (1, 16, 39):
        assert torch.equal(layer.forward_few(x[:t]), whole[:t])
    assert layer.forward_few(x[:0]).shape == (0, 256)


# up to and beyond the tokens that a workgroup routes for itself, the pairs
# that one wave tables, and tokens that a chunk's workgroup takes alone
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,kw", [
    (8, 192, 70, 8, {}), (13, 64, 70, 5, dict(n_bias=1)), (16, 128, 300, 4, dict(n_bias=2)),
    (17, 128, 300, 4, dict(n_bias=2)), (64, 4160, 90, 8, dict(n_bias=1)),
    (50, 256, 600, 3, dict(out=ops.OUT_BF16)), (21, 128, 40, 3, dict(mode=ops.MODE_HASH)),
    (22, 128, 40, 3, dict(mode=ops.MODE_HASH)), (64, 64, 1000, 8, dict(mode=ops.MODE_HASH))])
def test_routing_and_parts(T, d, E, k, kw, fp8):
    layer, w, x, ids, mod = make(T, d, E, k, 128, 64, fp8, T + d, **kw)
    whole = check(layer, w, x, ids, mod)
    for t in (1, T - 1):                             # alone and in the batch: the same bits
        cut = lambda v: None if v is None else v[:t]  # noqa: E731
        assert torch.equal(layer.forward_few(x[:t], input_ids=cut(ids), modality=cut(mod)),
                           whole[:t])


def test_hash_bad_ids_among_many():
    T, k = 60, 4
    layer, w, x, ids, _ = make(T, 128, 30, k, 64, 64, True, 19, mode=ops.MODE_HASH, V=20)
    table = layer.weights["tid2eid"]
    table[3] = torch.tensor([4, 9, 4, 9], dtype=torch.int32)
    table[5] = torch.tensor([1, 2, 30, 0], dtype=torch.int32)
    ids[7], ids[40], ids[59], ids[11] = 3, -5, 20, 5
    bad = (ids < 0) | (ids >= 20) | (ids == 5)
    got = torch.empty((T, k), dtype=torch.int32, device=DEV)
    wt = torch.empty((T, k), device=DEV)
    y = layer.forward_few(x, input_ids=ids, ids=got, w=wt)
    assert bool((got[bad] == -1).all()) and bool((wt[bad] == 0).all())
    assert torch.equal(got[~bad], table[ids[~bad].long()])
    assert ops.read_error_flags(layer.flags) == ops.FLAG_BAD_INPUT_ID | ops.FLAG_BAD_EXPERT_ID
    ref = plain(layer, w, x, got, wt)
    assert float((y.to(D) - ref).abs().max()) <= 1e-2 * float(ref.pow(2).mean().sqrt())


def test_equal_scores_take_the_lower_experts():
    layer, w, x, _, _ = make(4, 128, 70, 5, 64, 0, False, 8)
    layer.weights["w_g"].zero_()
    ids = torch.empty((4, 5), dtype=torch.int32, device=DEV)
    layer.forward_few(x, ids=ids)
    assert torch.equal(ids.cpu(), torch.arange(5, dtype=torch.int32).expand(4, 5))


@pytest.mark.parametrize("fp8", [False, True])
def test_hash_bad_ids_and_repeats(fp8):
    layer, w, x, ids, _ = make(12, 128, 10, 3, 64, 64, fp8, 9, mode=ops.MODE_HASH, V=20)
    table = layer.weights["tid2eid"]
    table[3] = torch.tensor([4, 4, 4], dtype=torch.int32)      # repeats: a row each
    table[5] = torch.tensor([1, 10, 2], dtype=torch.int32)     # out of range
    table[6] = torch.tensor([-1, 0, 2], dtype=torch.int32)
    ids.copy_(torch.tensor([3, 5, 6, -1, 20, 0, 3, 3, 1, 2, 4, 19], dtype=torch.int32))
    got = torch.empty((12, 3), dtype=torch.int32, device=DEV)
    wt = torch.empty((12, 3), device=DEV)
    y = layer.forward_few(x, input_ids=ids, ids=got, w=wt)
    assert bool((got[1:5] == -1).all()) and bool((wt[1:5] == 0).all())
    assert bool((got[0] == 4).all())
    assert ops.read_error_flags(layer.flags) == ops.FLAG_BAD_INPUT_ID | ops.FLAG_BAD_EXPERT_ID
    ref = plain(layer, w, x, got, wt)
    rms = float(ref.pow(2).mean().sqrt())
    assert float((y.to(D) - ref).abs().max()) <= 1e-2 * rms


@pytest.mark.parametrize("Fs", [0, 64])
def test_every_token_dropped(Fs):
    layer, w, x, ids, _ = make(3, 128, 10, 3, 64, Fs, False, 10, mode=ops.MODE_HASH, V=20)
    ids.fill_(99)
    got = torch.empty((3, 3), dtype=torch.int32, device=DEV)
    wt = torch.empty((3, 3), device=DEV)
    y = layer.forward_few(x, input_ids=ids, ids=got, w=wt)
    ref = plain(layer, w, x, got, wt)
    if Fs == 0:
        assert bool((y == 0).all())
    else:
        assert float((y.to(D) - ref).abs().max()) <= 1e-2 * float(ref.pow(2).mean().sqrt())


def test_many_rows_of_one_expert():
    """64 tokens whose table rows all name one expert 8 times: 512 rows."""
    layer, w, x, ids, _ = make(64, 128, 10, 8, 64, 0, False, 11, mode=ops.MODE_HASH, V=20)
    layer.weights["tid2eid"].fill_(7)
    got = torch.empty((64, 8), dtype=torch.int32, device=DEV)
    wt = torch.empty((64, 8), device=DEV)
    y = layer.forward_few(x, input_ids=ids, ids=got, w=wt)
    assert bool((got == 7).all())
    ref = ffn(layer, w, MATS[:3], 7, x.to(D)) * wt.to(D).sum(1, keepdim=True)
    assert float((y.to(D) - ref).abs().max()) <= 1e-2 * float(ref.pow(2).mean().sqrt())


def test_nan_token_stays_alone():
    layer, w, x, _, _ = make(5, 128, 16, 2, 64, 64, False, 12)
    clean = layer.forward_few(x)
    x2 = x.clone()
    x2[2, 77] = float("nan")
    y = layer.forward_few(x2)
    assert bool(torch.isnan(y[2]).all())
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("fp8", [False, True])
def test_workspace_of_any_content(fp8):
    layer, w, x, _, _ = make(9, 256, 24, 4, 192, 128, fp8, 13)
    y = layer.forward_few(x)
    layer.few_ws.fill_(0xff)
    assert torch.equal(layer.forward_few(x), y)


def test_matches_the_layer_forward():
    """The dispatch path on the same weights: one layer, two paths."""
    layer, w, x, _, _ = make(33, 512, 64, 6, 256, 256, False, 14)
    few, full = layer.forward_few(x), layer.forward(x)
    rms = float(full.pow(2).mean().sqrt())
    assert float((few - full).abs().max()) <= 1e-2 * rms


def test_refusals():
    layer, w, x, _, _ = make(8, 128, 8, 2, 64, 0, False, 15)
    with pytest.raises(ops.MoeError, match="at most 8 tokens"):
        layer.forward_few(torch.zeros((9, 128), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ops.MoeError, match="x must be"):
        layer.forward_few(torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV))
    packed = ops.MoeLayer(8, 128, 8, 2, 64, 0, w, packed=True)
    with pytest.raises(ops.MoeError, match="unsupported"):
        packed.forward_few(x)
    block, _, x, _, _ = make(8, 128, 8, 2, 64, 0, True, 16)
    with pytest.raises(ops.MoeError, match="unsupported"):
        block.forward(x)
    bad = dict(block.weights)
    bad["w_up_scale"] = bad["w_up_scale"].double()
    with pytest.raises(ops.MoeError, match="w_up_scale"):
        ops.MoeLayer(8, 128, 8, 2, 64, 0, bad, packed="fp8_block")


@pytest.mark.parametrize("fp8", [False, True])
def test_other_stream_and_graph(fp8):
    layer, w, x, _, _ = make(4, 256, 24, 4, 192, 128, fp8, 17)
    eager = layer.forward_few(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.empty_like(eager)
    with torch.cuda.stream(s):
        layer.forward_few(x, y=y)
    s.synchronize()
    assert torch.equal(y, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer.forward_few(x, y=y)
    for seed in (1, 2, 3):
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer.forward_few(x))
        torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_at_once_on_workspaces_of_their_own(fp8):
    """Two graphs of one layer, each with its own workspace, replayed on two
    streams beside each other, and an eager call on the layer's own beside
    both."""
    layer, w, x, _, _ = make(24, 512, 64, 6, 320, 256, fp8, 23)
    parts = [x[:5].clone(), x[5:].clone(), x[2:20].clone()]
    want = [layer.forward_few(p) for p in parts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [layer.few_workspace() for _ in range(2)]
    ys = [torch.empty_like(v) for v in want]
    graphs = []
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(8):
                layer.forward_few(parts[i], y=ys[i], ws=ws[i])
        graphs.append(graph)
    for _ in range(4):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for _ in range(8):
            layer.forward_few(parts[2], y=ys[2])
        torch.cuda.synchronize()
        for y, v in zip(ys, want):
            assert torch.equal(y, v)
    assert ops.read_error_flags(layer.flags) == 0
