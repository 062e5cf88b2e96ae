"""The operators around the layer and the MXFP4 ones on tensors of more than
2^31 values: a block of rows repeated, whose last copy has to come out as the
first."""
import pytest
import torch

from sparse_moe_layer_04_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def same_ends(t, rows):
    assert torch.equal(t[:rows], t[-rows:]) and t.numel() > 2 ** 31


def test_norm_and_backward():
    x = torch.randn(1000, 4096, device="cuda").bfloat16().repeat(530, 1)
    w = torch.randn(4096, device="cuda")
    _, y, codes, scales = ops.add_rms_norm(x, w, fp8=True)
    same_ends(y, 1000)
    same_ends(codes, 1000)
    assert torch.equal(scales[:1000], scales[-1000:])
    del codes
    dx, dw = ops.rms_norm_backward(x, w, y, dx_dtype=ops.OUT_BF16)
    same_ends(dx, 1000)
    one = ops.rms_norm_backward(x[:1000], w, y[:1000])[1].double() * 530
    # sums of 1036 rows a part in fp32
    assert ((dw.double() - one).abs() <= 1036 * 2.0 ** -24 *
            (y[:1000].double().abs() * 530 * 6).sum(0)).all()


def test_balance():
    lg = torch.randn(10000, 384, device="cuda").repeat(600, 1)
    ids = torch.rand(10000, 384, device="cuda").argsort(1)[:, :6].to(torch.int32).repeat(600, 1)
    off = (torch.arange(601) * 10000).to(torch.int32).cuda()
    loss, counts = ops.balance_loss(lg, ids, off)
    assert (counts == counts[:1]).all()
    assert ((loss / loss[0] - 1).abs() <= 64 * 2.0 ** -24).all()
    d = ops.balance_loss_backward(lg, ids, counts, torch.ones_like(loss), off)
    same_ends(d, 10000)
    assert d[-10000:].any()


def test_mxfp4():
    a = torch.randn(1000, 4096, device="cuda").bfloat16().repeat(530, 1)
    codes, scales = ops.quantize_mxfp4(a)
    assert a.numel() > 2 ** 31
    assert torch.equal(codes[:1000], codes[-1000:]) and torch.equal(scales[:1000], scales[-1000:])
    assert codes[-1000:].any()
    del a, codes
    a4 = torch.randint(0, 256, (1000, 32), dtype=torch.uint8, device="cuda").repeat(1100, 1)
    sa = torch.randint(120, 130, (1000, 2), dtype=torch.uint8, device="cuda").repeat(1100, 1)
    w4 = torch.randint(0, 256, (1, 2048, 32), dtype=torch.uint8, device="cuda")
    sw = torch.randint(120, 130, (1, 2048, 2), dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 1100000], dtype=torch.int32, device="cuda")
    out = ops.grouped_gemm_mxfp4(a4, sa, off, w4, sw, out_dtype=ops.OUT_F32)
    same_ends(out, 1000)
    assert out[-1000:].any()


def test_mxfp4_widest():
    """The most columns there may be, in tiles of 256 rows whose outputs end at
    2^32 bytes: the halves' products have the same bits."""
    N = 1 << 22
    draw = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    a4, sa = draw(0, 256, 512, 16), draw(120, 130, 512, 1)
    w4, sw = draw(0, 256, 1, N, 16), draw(120, 130, 1, N, 1)
    off = torch.tensor([0, 512], dtype=torch.int32, device="cuda")
    out = torch.full((512, N), -77.0, device="cuda")
    ops.grouped_gemm_mxfp4(a4, sa, off, w4, sw, out_dtype=ops.OUT_F32, out=out)
    for i in range(2):
        cols = slice(i * N // 2, (i + 1) * N // 2)
        half = ops.grouped_gemm_mxfp4(a4, sa, off, w4[:, cols].contiguous(),
                                      sw[:, cols].contiguous(), out_dtype=ops.OUT_F32)
        assert torch.equal(out[:, cols], half)
    assert out[-1].any()


def test_clip():
    n = 2 ** 31 + 4097
    g = torch.full((n,), 0.5, device="cuda")
    norm = ops.GradClip([g]).clip(1.0)
    assert abs(float(norm) / (0.5 * n ** 0.5) - 1) <= 1e-6
    want = 1.0 / n ** 0.5
    for part in (g[:5], g[2 ** 31 - 3:2 ** 31 + 5], g[-5:]):
        assert ((part.double() / want - 1).abs() <= 1e-6).all()


def test_mxfp4_most_rows():
    """As many rows as there may be, in one group: every 2^20 of them as the
    first ones, which are the 64-bit values, in bf16 what rounding leaves."""
    rows, part = (1 << 31) - 1, 1 << 20
    draw = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    first, scale = draw(0, 256, part, 16), draw(120, 130, part, 1)
    a4 = torch.empty(rows, 16, dtype=torch.uint8, device="cuda")
    sa = torch.empty(rows, 1, dtype=torch.uint8, device="cuda")
    for lo in range(0, rows, part):
        n = min(part, rows - lo)
        a4[lo:lo + n], sa[lo:lo + n] = first[:n], scale[:n]
    w4, sw = draw(0, 256, 1, 16, 16), draw(120, 130, 1, 16, 1)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out = torch.full((rows, 16), -77.0, dtype=torch.bfloat16, device="cuda")
    ops.grouped_gemm_mxfp4(a4, sa, off, w4, sw, out=out)
    assert out.numel() > 2 ** 31
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device="cuda")

    def of(c, s):
        v = value[torch.stack((c & 15, c >> 4), -1).flatten(-2).long()]
        return v * torch.exp2(s.double() - 127)
    a, w = of(first, scale), of(w4[0], sw[0])
    want, mag = a @ w.t(), a.abs() @ w.abs().t()
    got = out[:part].double()
    assert ((got - want).abs() <= 32 * 2.0 ** -24 * mag + want.abs() * 2.0 ** -8).all()
    for lo in range(0, rows, part):
        n = min(part, rows - lo)
        assert torch.equal(out[lo:lo + n], out[:n]), lo


def test_fp8_block_most_rows():
    """The 8-bit product in the same way."""
    rows, part = (1 << 31) - 1, 1 << 20
    first = torch.randint(0, 0x7f, (part, 16), dtype=torch.uint8, device="cuda")
    scale = torch.rand(part, 1, device="cuda") + 0.5
    a8 = torch.empty(rows, 16, dtype=torch.uint8, device="cuda")
    sa = torch.empty(rows, 1, device="cuda")
    for lo in range(0, rows, part):
        n = min(part, rows - lo)
        a8[lo:lo + n], sa[lo:lo + n] = first[:n], scale[:n]
    w8 = torch.randint(0, 0x7f, (1, 16, 16), dtype=torch.uint8, device="cuda")
    sw = torch.rand(1, 1, 1, device="cuda") + 0.5
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out = torch.full((rows, 16), -77.0, dtype=torch.bfloat16, device="cuda")
    ops.grouped_gemm_fp8_block(a8, sa, off, w8, sw, out=out)
    of = lambda c, s: c.view(torch.float8_e4m3fn).double() * s.double()  # noqa: E731
    want = of(first, scale) @ of(w8[0], sw[0]).t()
    got = out[:part].double()
    # values of one sign: 7 * 2^-13 of their sum at most is left out of a bf16
    # output's products, then one rounding
    assert ((got - want).abs() <= want * (2.0 ** -8 + 8 * 2.0 ** -13)).all()
    for lo in range(0, rows, part):
        n = min(part, rows - lo)
        assert torch.equal(out[lo:lo + n], out[:n]), lo


def test_balance_most_tokens():
    """As many tokens as there may be, 2047 times the same 2^20 and all but the
    last of them again as a second sequence, against 64 bits."""
    T, part, E = (1 << 31) - 1, 1 << 20, 2
    first = torch.randn(part, E, device="cuda")
    chosen = torch.randint(0, E, (part, 1), device="cuda").to(torch.int32)
    lg = torch.empty(T, E, device="cuda")
    ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    for lo in range(0, T, part):
        n = min(part, T - lo)
        lg[lo:lo + n], ids[lo:lo + n] = first[:n], chosen[:n]
    off = torch.tensor([0, 2047 * part, T], dtype=torch.int32, device="cuda")
    loss, counts = ops.balance_loss(lg, ids, off)
    d = ops.balance_loss_backward(lg, ids, counts, torch.ones_like(loss), off)
    s = torch.sigmoid(first.double())
    p = s / s.sum(1, keepdim=True)
    for seq, n in ((0, part), (1, part - 1)):
        times = 2047 if seq == 0 else 1
        c = torch.bincount(chosen[:n, 0].long(), minlength=E)
        assert torch.equal(counts[seq, 0].long(), c * times)
        f = c.double() * E / n
        q = p[:n] @ f
        # 64 steps of a row's sums and quotients, fp32 sums of 1024 tokens a wave
        assert abs(float(loss[seq, 0]) / float(q.mean()) - 1) <= (64 + 1024 + 8) * 2.0 ** -24
        up = p[:n] * (1 - s[:n]) / (n * times)
        at = seq * 2047 * part
        got = d[at:at + n].double()
        assert ((got - (f - q[:, None]) * up).abs() <= 64 * 2.0 ** -24 * (f + q[:, None]) * up).all()
    for i in range(1, 2047):
        assert torch.equal(d[i * part:(i + 1) * part], d[:part]), i
