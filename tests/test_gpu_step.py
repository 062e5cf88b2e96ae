"""GPU parity of the norm with the residual's addition, its backward, the
balance loss and its gradient, and the gradients' norm and clipping, against
the formulas in 64 bits (on the CPU).

Tolerances: a rounding is off by at most half a step (relative 2^-24 in fp32,
2^-8 in bf16 counted by torch.finfo(t).eps / 2, and half the least subnormal);
the sums of the norm and of the gradients' norm are held in 64 bits (relative
2^-40 covers them); fp32 sums of n terms are off by at most n 2^-24 of the sum
of their magnitudes."""
import math

import numpy as np
import pytest
import torch

from sparse_moe_layer_04_amd import ops

pytestmark = pytest.mark.gpu
D = torch.float64
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134}


def near(got, want, tol, what):
    """|got - want| <= tol, element by element, and the same NaN."""
    got, want = got.cpu().to(D), want.to(D)
    assert torch.equal(got.isnan(), want.isnan()), what
    bad = ~((got - want).abs() <= tol) & ~want.isnan() & (got != want)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4])


def rounded(want, dt, more=0.0):
    """Tolerance of one rounding to dt of a value known to within `more`."""
    return want.abs() * HALF[dt] * (1 + 2.0 ** -20) + TINY[dt] + more


# ------------------------------------------------------------------- norm --
def norm_inputs(rows, d, xt, rt, wt, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + rows * 7 + d)
    x = (torch.randn(rows, d, generator=g) * scale).to(xt)
    r = None if rt is None else (3 * scale * torch.randn(rows, d, generator=g)).to(rt)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(wt)
    return x, r, w


def norm_ref(x, r, w, eps):
    s = x
    if r is not None:
        s = (x.float() + r.float()).to(r.dtype)     # fp32 sum, one rounding
    v = s.to(D)
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return s, n * w.to(D)


def block_scales(y):
    """The least powers of two with max|y| <= 448 * scale, 128 values each."""
    rows, d = y.shape
    b = torch.nn.functional.pad(y, (0, -d % 128)).view(rows, -1, 128).abs().amax(2)
    m, e = torch.frexp(b)
    return torch.where(b > 0, torch.exp2((e - torch.where(m <= 0.875, 9, 8)).to(D).clamp(-126, 120)),
                       torch.ones_like(b)), b


def check_norm(x, r, w, eps=1e-6, fp8=True, want_y=True, inplace=False):
    s_ref, y_ref = norm_ref(x, r, w, eps)
    dx, dr, dw = x.cuda(), None if r is None else r.cuda(), w.cuda()
    s, y, codes, scales = ops.add_rms_norm(dx, dw, residual=dr, eps=eps, fp8=fp8, want_y=want_y,
                                           res=dr if inplace else None)
    torch.cuda.synchronize()
    if r is None:
        assert s is dx and torch.equal(s.cpu(), x)
    else:
        assert s.dtype == r.dtype and torch.equal(s.cpu(), s_ref)
        assert not inplace or s is dr
    two = y_ref.abs() * 2.0 ** -22      # n and n w rounded to fp32
    if want_y:
        near(y, y_ref, rounded(y_ref, BF16, two), "y")
    else:
        assert y is None
    if not fp8:
        assert codes is None and scales is None
        return
    want, amax = block_scales(y_ref)
    sc = scales.cpu().to(D)
    border = (amax / want / 448 - 1).abs() < 2.0 ** -20     # (of 448 2^X, either side)
    border |= (amax / want / 224 - 1).abs() < 2.0 ** -20
    assert torch.all((sc == want) | border)
    full = sc.repeat_interleave(128, 1)[:, :x.shape[1]]
    q = codes.cpu().view(torch.float8_e4m3fn).to(D) * full
    tol = torch.maximum(y_ref.abs() * 2.0 ** -4, full * 2.0 ** -10) * (1 + 2.0 ** -18) + two
    near(q, y_ref, tol, "codes")


@pytest.mark.parametrize("d", [16, 64, 112, 128, 144, 512, 528, 1024, 2000, 4096, 4112, 8192,
                               9008, 16384])
@pytest.mark.parametrize("rows", [1, 3, 1029])
def test_norm_sizes(rows, d):
    if rows > 100 and d > 8192:
        rows = 65
    check_norm(*norm_inputs(rows, d, BF16, BF16, F32))


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("wt", [BF16, F32])
def test_norm_types(xt, rt, wt):
    check_norm(*norm_inputs(7, 1040, xt, rt, wt))
    check_norm(*norm_inputs(1100, 272, xt, rt, wt), want_y=False)
    check_norm(*norm_inputs(5, 2056, xt, rt, wt), fp8=False)
    check_norm(*norm_inputs(5, 8, xt, rt, wt), fp8=False)


@pytest.mark.parametrize("rt", [BF16, F32])
def test_norm_in_place(rt):
    check_norm(*norm_inputs(33, 4096, BF16, rt, BF16), inplace=True)
    check_norm(*norm_inputs(2049, 528, BF16, rt, BF16), inplace=True)


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 1e37])
def test_norm_magnitudes(scale):
    """Sums of squares far outside fp32."""
    x, _, w = norm_inputs(5, 512, F32, None, F32, scale=scale)
    check_norm(x, None, w, eps=0.0)
    check_norm(x, None, w, eps=1e-6)


def test_norm_zero_rows_and_values():
    x, r, w = norm_inputs(6, 256, BF16, BF16, F32)
    x[2], r[2] = 0, 0
    w[128:] = 0
    check_norm(x, r, w)
    s, y, c, sc = ops.add_rms_norm(x[:0].cuda(), w.cuda(), residual=r[:0].cuda(), fp8=True)
    assert s.shape == (0, 256) and y.shape == (0, 256) and sc.shape == (0, 2)


def test_norm_not_finite():
    """NaN and infinities stay in their rows; their codes are NaN."""
    x, _, w = norm_inputs(5, 256, F32, None, F32)
    x[1, 3], x[3, 200] = float("nan"), float("inf")
    _, y, c, sc = ops.add_rms_norm(x.cuda(), w.cuda(), fp8=True)
    y, v = y.cpu(), c.cpu().view(torch.float8_e4m3fn).float()
    assert y[1].isnan().all() and v[1].isnan().all()
    assert y[3, 200].isnan() and v[3, 200].isnan()
    keep = [0, 2, 4]
    _, y2, c2, sc2 = ops.add_rms_norm(x[keep].cuda(), w.cuda(), fp8=True)
    assert torch.equal(y[keep], y2.cpu()) and torch.equal(c.cpu()[keep], c2.cpu())
    assert torch.equal(sc.cpu()[keep], sc2.cpu()) and torch.equal(sc.cpu()[1], torch.ones(2))


def test_norm_rows_apart():
    """A row has the same bits alone and among many (another split of its sum)."""
    x, r, w = norm_inputs(1500, 2064, BF16, F32, BF16)
    many = ops.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), fp8=True)
    few = ops.add_rms_norm(x[7:9].cuda(), w.cuda(), residual=r[7:9].cuda(), fp8=True)
    for a, b in zip(many, few):
        assert torch.equal(a[7:9], b)


# ---------------------------------------------------------- norm backward --
def backward_ref(s, w, dy, d_res, eps):
    s, w, dy = s.to(D), w.to(D), dy.to(D)
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    n, g = s * r, dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    mag = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if d_res is not None:
        dx, mag = dx + d_res.to(D), mag + d_res.to(D).abs()
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def check_backward(rows, d, st=F32, wt=F32, gt=F32, rt=F32, xt=F32, eps=1e-6, seed=1):
    s, _, w = norm_inputs(rows, d, st, None, wt, seed=seed)
    g = torch.Generator().manual_seed(rows + 5 * d)
    dy = torch.randn(rows, d, generator=g).to(gt)
    d_res = None if rt is None else torch.randn(rows, d, generator=g).to(rt)
    dx, dw, mag, dmag = backward_ref(s, w, dy, d_res, eps)
    got, gw = ops.rms_norm_backward(s.cuda(), w.cuda(), dy.cuda(), eps=eps,
                                    d_res=None if d_res is None else d_res.cuda(),
                                    dx_dtype=ops.OUT_F32 if xt == F32 else ops.OUT_BF16)
    assert got.dtype == xt and gw.dtype == F32
    # the row's sums and terms in 64 bits, one rounding; dw: n rounded, then
    # an fp32 sum of at most `rows` terms
    near(got, dx, rounded(dx, xt, mag * 2.0 ** -40), "dx")
    near(gw, dw, (rows + 2) * 2.0 ** -24 * dmag + TINY[F32], "dw")


@pytest.mark.parametrize("d", [8, 64, 520, 1024, 1032, 2056, 4096, 4104, 8192, 9000, 16384])
@pytest.mark.parametrize("rows", [1, 5, 1031])
def test_backward_sizes(rows, d):
    check_backward(min(rows, 67) if d > 8192 else rows, d)


@pytest.mark.parametrize("st", [BF16, F32])
@pytest.mark.parametrize("gt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_backward_types(st, gt, rt, xt):
    check_backward(9, 1040, st, BF16, gt, rt, xt)
    check_backward(70, 264, st, F32, gt, rt, xt, eps=1e-2)


def test_backward_no_rows():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    dw = torch.full((64,), 7.0, device="cuda")
    dx, dw = ops.rms_norm_backward(e, w, e, dw=dw)
    assert dx.shape == (0, 64) and torch.equal(dw.cpu(), torch.zeros(64))


def test_backward_in_place_and_twice():
    s, r, w = norm_inputs(100, 528, F32, F32, F32)
    dy, res = torch.randn(100, 528).cuda(), torch.randn(100, 528).cuda()
    a = ops.rms_norm_backward(s.cuda(), w.cuda(), dy, d_res=res)
    b = ops.rms_norm_backward(s.cuda(), w.cuda(), dy, d_res=res)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = ops.rms_norm_backward(s.cuda(), w.cuda(), dy.clone(), d_res=res, dx=res)
    assert c[0] is res and torch.equal(c[0], a[0])


def test_backward_against_differences():
    """dx and dw against central differences of the forward's formula."""
    s, _, w = norm_inputs(3, 24, F32, None, F32)
    c = torch.randn(3, 24, dtype=D)
    f = lambda s, w: float((norm_ref(s, None, w, 1e-3)[1] * c).sum())  # noqa: E731
    dx, dw = ops.rms_norm_backward(s.cuda(), w.cuda(), c.float().cuda(), eps=1e-3)
    c = c.float().to(D)
    h = 1e-5
    for i in range(3):
        for j in range(0, 24, 5):
            e = torch.zeros(3, 24, dtype=D)
            e[i, j] = h
            d = (f(s.to(D) + e, w) - f(s.to(D) - e, w)) / (2 * h)
            # the third derivative's part of the difference: below 1e-7 here
            assert abs(float(dx[i, j]) - d) <= 1e-6 * (1 + abs(d))
    for j in range(24):
        e = torch.zeros(24, dtype=D)
        e[j] = h
        d = (f(s, w.to(D) + e) - f(s, w.to(D) - e)) / (2 * h)
        assert abs(float(dw[j]) - d) <= 1e-6 * (1 + abs(d))


# ---------------------------------------------------------------- balance --
def balance_inputs(T, E, k, S, classes, masked=0.0, bad=0, seed=0, spread=1.5, offsets=None):
    rng = np.random.default_rng(seed + T * 3 + E)
    logits = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32))
    ids = torch.from_numpy(np.argsort(-rng.random((T, E)), axis=1)[:, :k].astype(np.int32))
    if k > E:
        ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32))
    ids = ids.contiguous()
    if offsets is None:
        cuts = np.sort(rng.integers(0, T + 1, S - 1)) if S > 1 else np.zeros(0, int)
        offsets = np.concatenate([[0], cuts, [T]])
    off = torch.tensor(np.asarray(offsets, np.int32))
    mod = torch.from_numpy((rng.random(T) < 0.4).astype(np.uint8) * 3) if classes == 2 else None
    mask = torch.from_numpy((rng.random(T) >= masked).astype(np.uint8)) if masked else None
    for t in range(0, T, max(1, T // bad)) if bad else ():
        ids[t, t % k] = (-1, E, 1 << 30)[t % 3]
    return logits, ids, off, mod, mask


def balance_ref(logits, ids, off, mod, mask, d_loss=None):
    """(loss, counts, d_logits, tolerance of d_logits) in 64 bits."""
    T, E = logits.shape
    k, S, C = ids.shape[1], len(off) - 1, 1 if mod is None else 2
    loss, counts = torch.zeros(S, C, dtype=D), torch.zeros(S, C, E, dtype=torch.int32)
    d, mag = torch.zeros(T, E, dtype=D), torch.zeros(T, E, dtype=D)
    ok = ((ids >= 0) & (ids < E)).all(1)
    if mask is not None:
        ok &= mask != 0
    o = [min(max(int(v), 0), T) for v in off]
    for i in range(S):
        for j in range(C):
            t = torch.arange(o[i], o[i + 1])
            t = t[ok[t]]
            if mod is not None:
                t = t[(mod[t] != 0) == bool(j)]
            if not len(t):
                continue
            z = logits[t].to(D).clamp(-80, 80)
            s, ns = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
            p = s / s.sum(1, keepdim=True)
            c = torch.bincount(ids[t].reshape(-1).long(), minlength=E)
            f = c.to(D) * E / (k * len(t))
            q = p @ f
            counts[i, j], loss[i, j] = c.to(torch.int32), q.mean()
            if d_loss is not None:
                up = d_loss[i, j].to(D) / len(t)
                d[t] = up * (f - q[:, None]) * p * ns
                mag[t] = up.abs() * (f + q[:, None]) * p * ns
    return loss, counts, d, mag


# a score is within 4 steps of S, its sums over E <= 1024 experts have at most
# 16 + 6 additions on the way of a term, quotients and products a step each:
# under 64 steps for q and for the gradient's factors
STEPS = 64 * 2.0 ** -24


def check_balance(T, E, k, S, classes, masked=0.0, bad=0, use_offsets=True, add=False, **kw):
    logits, ids, off, mod, mask = balance_inputs(T, E, k, S, classes, masked, bad, **kw)
    if not use_offsets:
        off = torch.tensor([0, T], dtype=torch.int32)
    S, C = len(off) - 1, classes
    d_loss = torch.randn(S, C, generator=torch.Generator().manual_seed(T))
    loss, counts, d, mag = balance_ref(logits, ids, off, mod, mask, d_loss)
    cu = lambda v: None if v is None else v.cuda()  # noqa: E731
    where = dict(offsets=off.cuda() if use_offsets else None, modality=cu(mod), mask=cu(mask))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    lg, di = logits.cuda(), ids.cuda()
    gl, gc = ops.balance_loss(lg, di, flags=flags, **where)
    assert gl.shape == (S, C) and torch.equal(gc.cpu(), counts)
    near(gl, loss, loss * STEPS, "loss")
    base = torch.randn(T, E) if add else None
    gd = ops.balance_loss_backward(lg, di, gc, d_loss.cuda(), add=cu(base), **where)
    want, tol = d, mag * STEPS + TINY[F32] * 4
    if add:
        want = d + base.to(D)
        tol = tol + want.abs() * 2.0 ** -24
    near(gd, want, tol, "d_logits")
    in_seq = torch.zeros(T, dtype=torch.bool)
    in_seq[max(0, int(off[0])):max(0, min(T, int(off[-1])))] = True
    live = in_seq if mask is None else in_seq & (mask != 0)
    dropped = ((ids < 0) | (ids >= E)).any(1) & live
    assert ops.read_error_flags(flags) == (ops.FLAG_BAD_EXPERT_ID if dropped.any() else 0)
    return lg, di, where, gl, gc


@pytest.mark.parametrize("T", [1, 2, 65, 1024, 1025, 3001])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (63, 3), (64, 6), (130, 8), (384, 6), (500, 1),
                                 (1024, 8)])
def test_balance_sizes(T, E, k):
    check_balance(T, E, k, 1, 1, use_offsets=T % 2 == 0)
    check_balance(T, E, k, min(T, 5), 2)


@pytest.mark.parametrize("T,S", [(40, 64), (300, 300), (4000, 7), (5000, 200), (2500, 1200)])
@pytest.mark.parametrize("masked,bad", [(0.0, 0), (0.3, 0), (0.0, 5), (0.3, 40)])
def test_balance_sequences(T, S, masked, bad):
    """Many sequences, empty and of one token; masked tokens; ids out of range."""
    check_balance(T, 72, 4, S, 2, masked, bad)
    check_balance(T, 50, 2, S, 1, masked, bad, add=True)


@pytest.mark.parametrize("T,offsets", [
    (100, [0, 0, 0]), (100, [100, 100]), (100, [10, 30, 90]), (2100, [1030, 1031, 2090]),
    (100, [-5, 50, 1000]), (2100, [2050, 2060]), (1500, [0, 10])])
def test_balance_offsets(T, offsets):
    """Tokens outside every sequence, offsets outside [0, T]."""
    check_balance(T, 40, 3, None, 2, offsets=offsets)


def test_balance_all_masked():
    """Groups without a token: loss 0, counts 0, gradient 0."""
    lg, ids, off, mod, _ = balance_inputs(70, 20, 2, 3, 2)
    mask = torch.zeros(70, dtype=torch.uint8).cuda()
    loss, counts = ops.balance_loss(lg.cuda(), ids.cuda(), off.cuda(), mod.cuda(), mask)
    assert not loss.any() and not counts.any()
    d = ops.balance_loss_backward(lg.cuda(), ids.cuda(), counts, torch.ones_like(loss), off.cuda(),
                                  mod.cuda(), mask)
    assert not d.any() and not d.isnan().any()
    empty = ops.balance_loss(lg[:0].cuda(), ids[:0].cuda())
    assert empty[0].tolist() == [[0.0]] and not empty[1].any() and empty[1].shape == (1, 1, 20)


@pytest.mark.parametrize("spread", [1e-3, 20.0, 60.0])
def test_balance_saturated(spread):
    """Scores next to 1 and to 0: 1 - S and the row sums keep their bits."""
    check_balance(200, 96, 4, 3, 1, spread=spread)


def test_balance_repeated_expert():
    """A hash table may name an expert twice, and fewer experts than slots."""
    check_balance(129, 5, 8, 2, 1)


def test_balance_even_load():
    """Equal logits: the loss is 1 whatever the routes, its gradient 0 in sum."""
    lg = torch.zeros(96, 12, device="cuda")
    ids = (torch.arange(96 * 3) % 12).view(96, 3).to(torch.int32).cuda()
    loss, counts = ops.balance_loss(lg, ids)
    assert abs(float(loss) - 1) <= STEPS and counts.unique().tolist() == [24]


def test_balance_add_in_place_and_same_bits():
    lg, ids, where, loss, counts = check_balance(3000, 128, 6, 9, 2)
    again = ops.balance_loss(lg, ids, **where)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)
    base = torch.randn(3000, 128, device="cuda")
    dl = torch.ones_like(loss)
    a = ops.balance_loss_backward(lg, ids, counts, dl, add=base, **where)
    b = ops.balance_loss_backward(lg, ids, counts, dl, add=base, out=base, **where)
    assert b is base and torch.equal(a, b)


def test_balance_against_differences():
    lg, ids, off, mod, mask = balance_inputs(12, 7, 2, 2, 2, masked=0.2)
    dl = torch.tensor([[0.3, -0.7], [1.0, 0.5]])
    cu = [v.cuda() for v in (lg, ids, off, mod, mask)]
    _, counts = ops.balance_loss(*cu)
    d = ops.balance_loss_backward(cu[0], cu[1], counts, dl.cuda(), *cu[2:])
    f = lambda z: float((balance_ref(z, ids, off, mod, mask)[0] * dl.to(D)).sum())  # noqa: E731
    h = 1e-5
    for t in range(12):
        for j in range(7):
            e = torch.zeros(12, 7, dtype=D)
            e[t, j] = h
            want = (f(lg.to(D) + e) - f(lg.to(D) - e)) / (2 * h)
            assert abs(float(d[t, j]) - want) <= 1e-6


# ------------------------------------------------------------------- clip --
def clip_case(sizes, types, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + len(sizes))
    return [(torch.randn(n, generator=g) * scale).to(t) for n, t in zip(sizes, types)]


def clip_ref(grads, max_norm):
    n = math.sqrt(math.fsum(float((g.to(D) ** 2).sum()) for g in grads))
    return n, max_norm / n if n > max_norm else 1.0


SIZES = [[1], [7, 8192, 1], [8191, 8193, 3, 65536, 40000], [1 << 20, 5, 300001],
         list(range(1, 300))]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("place", ["in place", "apart"])
def test_clip(sizes, kind, place):
    types = [F32 if kind == "f32" or (kind == "mixed" and i % 2) else BF16
             for i in range(len(sizes))]
    grads = clip_case(sizes, types)
    for share in (0.37, 2.0):
        n, _ = clip_ref(grads, 1.0)
        max_norm = n * share
        _, f = clip_ref(grads, max_norm)
        dev = [g.cuda() for g in grads]
        out = [torch.full_like(g, 9.0) for g in dev] if place == "apart" else None
        c = ops.GradClip(dev, out=out)
        first = c.norm()
        norm = c.clip(max_norm)
        assert torch.equal(first, norm)
        near(norm, torch.tensor([n], dtype=D), n * 2.0 ** -23, "norm")
        for g, d, o in zip(grads, dev, c.out):
            want = g.to(D) * f
            near(o, want, 0.0 if f == 1.0 else rounded(want, g.dtype), "clipped")
            if place == "apart":
                assert torch.equal(d.cpu(), g)
        if place == "in place" and f < 1:
            now = float(c.norm())
            assert abs(now / max_norm - 1) <= 2.0 ** -7


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e25, 2e38])
def test_clip_magnitudes(scale):
    """Squares far outside fp32; a norm outside fp32 is inf and clips all the same."""
    grads = [g.clamp(-1.5 * scale, 1.5 * scale) for g in clip_case([5000, 9000], [F32, F32], scale)]
    n, f = clip_ref(grads, 1e-3 * scale)
    dev = [g.cuda() for g in grads]
    norm = ops.GradClip(dev).clip(1e-3 * scale)
    near(norm, torch.tensor([n], dtype=D).float(), n * 2.0 ** -22, "norm")
    for g, d in zip(grads, dev):
        near(d, g.to(D) * f, rounded(g.to(D) * f, F32), "clipped")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 8191, 12345, 20000 - 1])
def test_clip_not_finite(value, at):
    """A gradient that is not finite: the norm says so, nothing is scaled."""
    grads = clip_case([20000, 100], [F32, BF16])
    grads[0][at] = value
    dev = [g.cuda() for g in grads]
    norm = ops.GradClip(dev).clip(1e-3)
    assert not torch.isfinite(norm).any()
    for g, d in zip(grads, dev):
        assert torch.equal(torch.nan_to_num(d.cpu(), nan=7.0), torch.nan_to_num(g, nan=7.0))


def test_clip_limits():
    """Zero gradients, max_norm 0 and inf, tensors without values, of several dims."""
    z = [torch.zeros(3, 5, device="cuda"), torch.zeros(0, 4, device="cuda")]
    assert ops.GradClip(z).clip(1.0).tolist() == [0.0] and not z[0].any()
    assert ops.GradClip([torch.zeros(0, device="cuda")]).clip(1.0).tolist() == [0.0]
    g = torch.randn(4, 5, 6, device="cuda")
    keep = g.clone()
    ops.GradClip([g]).clip(float("inf"))
    assert torch.equal(g, keep)
    ops.GradClip([g]).clip(0.0)
    assert not g.any()


def test_refusals():
    """What the binding refuses with tensors on the device."""
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    loss, counts = ops.balance_loss(x, ids)
    for call in (lambda: ops.add_rms_norm(x.half(), w), lambda: ops.add_rms_norm(x, w[:32]),
                 lambda: ops.add_rms_norm(x.t(), w), lambda: ops.add_rms_norm(x, w.cpu()),
                 lambda: ops.add_rms_norm(x, w, residual=x[:4]),
                 lambda: ops.add_rms_norm(x, w, res=x), lambda: ops.add_rms_norm(x[0], w),
                 lambda: ops.add_rms_norm(x, w, want_y=False),
                 lambda: ops.add_rms_norm(x, w, residual=x, res=x.to(BF16)),
                 lambda: ops.add_rms_norm(x, w, eps=-1.0),
                 lambda: ops.add_rms_norm(x[:, :12].contiguous(), w[:12]),
                 lambda: ops.rms_norm_backward(x, w, x[:, :32]),
                 lambda: ops.rms_norm_backward(x, w, x, dx=x.to(BF16)),
                 lambda: ops.rms_norm_backward(x, w, x, workspace=torch.empty(
                     8, dtype=torch.uint8, device="cuda")),
                 lambda: ops.balance_loss(x, ids.long()), lambda: ops.balance_loss(x, ids[:4]),
                 lambda: ops.balance_loss(x, ids, offsets=ids[:1, :1].reshape(-1)),
                 lambda: ops.balance_loss(x, ids, mask=torch.ones(8, device="cuda")),
                 lambda: ops.balance_loss_backward(x, ids, counts[0], loss),
                 lambda: ops.balance_loss_backward(x, ids, counts, loss, add=x[:4]),
                 lambda: ops.balance_loss_backward(x, ids, counts, loss.double())):
        with pytest.raises(ops.MoeError):
            call()


def test_clip_refuses():
    a = torch.randn(64, device="cuda")
    for grads, out in (([a, a], None), ([a, a[16:32]], None), ([a], [torch.zeros(63).cuda()]),
                       ([a], [torch.zeros(64, dtype=BF16).cuda()]), ([a[1:]], None),
                       ([a[::2]], None), ([a.half()], None), ([a, a.clone()], [a.clone(), a])):
        with pytest.raises(ops.MoeError):
            ops.GradClip(grads, out=out)
    with pytest.raises(ops.MoeError):
        ops.GradClip([a]).clip(-1.0)
    with pytest.raises(ops.MoeError):
        ops.GradClip([a]).clip(float("nan"))


# ------------------------------------------------------- graphs, streams --
def replays(call, again, outs, rounds=3):
    """Every replay of a captured call gives what the eager call gives."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(rounds):
        again(i)
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        again(i)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_graph_replays():
    T, d, E, k = 1300, 512, 96, 4
    x, res = torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda")
    w = torch.rand(d, device="cuda")
    s, y = torch.empty_like(res), torch.empty(T, d, dtype=BF16, device="cuda")
    codes = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, 4, device="cuda")
    dx, dw = torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
    nws = torch.empty(ops.rms_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    lg, ids = torch.empty(T, E, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 700, 1200, 1300], dtype=torch.int32, device="cuda")
    loss, counts = torch.empty(3, 1, device="cuda"), torch.empty(3, 1, E, dtype=torch.int32,
                                                                 device="cuda")
    bws = torch.empty(ops.balance_loss_workspace_size(T, E, 3), dtype=torch.uint8, device="cuda")
    dl, dlg = torch.ones(3, 1, device="cuda"), torch.empty(T, E, device="cuda")
    clipped = [torch.empty_like(dx), torch.empty_like(dw)]
    clip, norm = ops.GradClip([dx, dw], out=clipped), torch.empty(1, device="cuda")

    def again(i):
        g = torch.Generator(device="cuda").manual_seed(i)
        x.normal_(generator=g)
        res.normal_(generator=g)
        lg.normal_(generator=g)
        ids.copy_(torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k])

    def call():
        ops.add_rms_norm(x, w, residual=res, fp8=True, res=s, y=y, codes=codes, scales=scales)
        ops.rms_norm_backward(s, w, x, d_res=res, dx=dx, dw=dw, workspace=nws)
        ops.balance_loss(lg, ids, off, loss=loss, counts=counts, workspace=bws)
        ops.balance_loss_backward(lg, ids, counts, dl, off, out=dlg)
        clip.clip(1.0, norm=norm)
    again(0)
    replays(call, again, [s, y, codes, scales, dx, dw, loss, counts, dlg, norm] + clipped)


def test_another_stream():
    """Calls go to the current stream, with inputs made on it."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x = torch.randn(64, 1024, device="cuda")
        s, y, _, _ = ops.add_rms_norm(x, torch.ones(1024, device="cuda"))
        c = ops.GradClip([x])
        n = c.norm()
    side.synchronize()
    xs = x.cpu()
    _, want = norm_ref(xs, None, torch.ones(1024), 1e-6)
    near(y, want, rounded(want, BF16, want.abs() * 2.0 ** -22), "y")
    assert abs(float(n) / float(xs.to(D).norm()) - 1) < 1e-6


@pytest.mark.parametrize("E,k", [(1, 1), (8, 1), (100, 3)])
@pytest.mark.parametrize("d_loss", [1.0, 65536.0, 1e8])
def test_balance_gradient_of_small_scores(E, k, d_loss):
    """Logits at the clamp's lower end, where a row's scores add up to 1e-33, with
    a scaled loss: the gradient is of the order of d_loss / T_g all the same."""
    g = torch.Generator().manual_seed(E)
    lg = -81 + 3 * torch.rand(3, E, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(3)]).to(torch.int32)
    off = torch.tensor([0, 1, 3], dtype=torch.int32)
    dl = torch.full((2, 1), d_loss)
    _, counts, d, mag = balance_ref(lg, ids, off, None, None, dl)
    got = ops.balance_loss_backward(lg.cuda(), ids.cuda(), counts.cuda(), dl.cuda(), off.cuda())
    near(got, d, mag * STEPS + TINY[F32] * 4, "d_logits")


@pytest.mark.parametrize("d", [8, 520, 1024, 4104, 9000])
@pytest.mark.parametrize("gt", [BF16, F32])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_backward_not_finite(d, gt, value):
    """An infinity or NaN in a row's first gradients: what the formula makes of
    it, whatever the row's width, in its row alone."""
    s, _, w = norm_inputs(6, d, F32, None, F32)
    dy = torch.randn(6, d, generator=torch.Generator().manual_seed(d)).to(gt)
    dy[1, 0], dy[4, 5] = value, -value
    dx, dw, mag, dmag = backward_ref(s, w, dy, None, 1e-6)
    got, gw = ops.rms_norm_backward(s.cuda(), w.cuda(), dy.cuda())
    near(got, dx, rounded(dx, F32, mag * 2.0 ** -40), "dx")
    near(gw, dw, 8 * 2.0 ** -24 * dmag + TINY[F32], "dw")


@pytest.mark.parametrize("rows,d", [(1 << 24, 8), (1 << 21, 520)])
def test_backward_many_rows(rows, d):
    """dw of many rows of one sign, whose terms end in bits that a long fp32 sum
    does not hold: fp32 sums of 512 rows at most, the rest in 64 bits."""
    s = torch.ones(1, d, dtype=BF16, device="cuda").expand(rows, d).contiguous()
    dy = torch.full((rows, d), 1 + 0.4 * 2.0 ** -10, device="cuda")
    dw = ops.rms_norm_backward(s, torch.ones(d, device="cuda"), dy, eps=0.0,
                               dx_dtype=ops.OUT_BF16)[1]
    want = torch.full((d,), float(dy[0, 0].double()) * rows, dtype=D)
    near(dw, want, want * (512 + 1) * 2.0 ** -24, "dw")


@pytest.mark.parametrize("rows,d", [(524288 + 1, 8), (262144 + 515, 2056)])
@pytest.mark.parametrize("inplace", [False, True])
def test_backward_in_several_launches(rows, d, inplace):
    """More rows than one launch takes: dx has the bits of its parts' calls, dw is
    the 64-bit sum."""
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s, dy, res = (draw(rows, d).to(BF16) for _ in range(3))
    w = draw(d)
    cuts = [0, 1000, rows - 700, rows]
    parts = [ops.rms_norm_backward(s[a:b], w, dy[a:b], d_res=res[a:b], dx_dtype=ops.OUT_BF16)[0]
             for a, b in zip(cuts, cuts[1:])]
    dw, mag = torch.zeros(d, dtype=D, device="cuda"), torch.zeros(d, dtype=D, device="cuda")
    for a in range(0, rows, 1 << 16):
        v = s[a:a + (1 << 16)].to(D)
        t = dy[a:a + (1 << 16)].to(D) * v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
        dw, mag = dw + t.sum(0), mag + t.abs().sum(0)
    got, gw = ops.rms_norm_backward(s, w, dy, d_res=res, dx_dtype=ops.OUT_BF16,
                                    dx=dy if inplace else None)
    assert torch.equal(got, torch.cat(parts))
    near(gw, dw.cpu(), ((512 + 2) * 2.0 ** -24 * mag).cpu() + TINY[F32], "dw")
