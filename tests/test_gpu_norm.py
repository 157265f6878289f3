"""Root-mean-square norm with the residual on the GPU, 16-bit and block outputs and the backward
pass, against the formula in 64 bits (block_reference.py)."""
import pytest
import torch

from block_reference import HALF, TINY, blocks, norm, rows_of

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    with T.Context(0) as c:
        yield c


def gain_of(cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    host = (1.0 + 0.2 * torch.randn(cols, generator=g)).to(dtype)
    return host.cuda(), host


# Roundings of binary32 on the way to y: a square's sum passes fewer than 140 additions (a lane's
# own, then lanes and waves; rows of over 16,384 columns: cols / 1,024 more), halved by the square
# root; seven more for the mean, eps, root, quotient, two products and s.
def f32_error(cols):
    return (77 + cols / 2048) * 2.0 ** -24


SIZES = [(1, 1), (2, 7), (3, 64), (5, 129), (4, 512), (9, 513), (3, 1000), (2, 1024), (7, 1408),
         (2, 2049), (3, 4096), (2, 5000), (1, 8192), (2, 9001), (1, 16384), (2, 16385), (1, 40000)]


@pytest.mark.parametrize("dtype,gain_dtype", [(BF, BF), (F16, F16), (BF, F32), (F16, F32)])
@pytest.mark.parametrize("n,cols", SIZES)
def test_norm(ctx, n, cols, dtype, gain_dtype):
    x, hx = rows_of(n, cols, dtype, cols)
    r, hr = rows_of(n, cols, dtype, cols + 1, spread=3.0)
    gain, hg = gain_of(cols, gain_dtype, cols + 2)
    e = f32_error(cols)

    def check(y, want):
        tol = want.abs() * (HALF[dtype] * (1 + 2 * e) + e) + TINY[dtype]
        assert ((y.cpu().double() - want).abs() <= tol).all()

    check(ctx.rms_norm(x, gain, EPS), norm(hx, hg, EPS)[0])
    y, total = ctx.rms_norm(x, gain, EPS, residual=r)
    s = hx.float() + hr.float()
    want, _ = norm(s, hg, EPS)
    check(y, want)
    assert torch.equal(total.cpu(), s.to(dtype))
    b, total = ctx.rms_norm(x, gain, EPS, residual=r, blocks=True)
    assert torch.equal(total.cpu(), s.to(dtype))
    assert b.q.shape == (n, cols) and b.scale.shape == (n, blocks(cols))
    wide = torch.zeros(n, 128 * blocks(cols), dtype=torch.float64)
    wide[:, :cols] = want
    big = wide.reshape(n, -1, 128).abs().amax(dim=2)
    scale = b.scale.cpu().double()
    # the largest is off by e, the scale by one rounding more
    assert ((scale - (big / 448).clamp(min=2.0 ** -126)).abs() <= (e + 2.0 ** -23) * scale).all()
    s128 = scale.repeat_interleave(128, dim=1)[:, :cols]
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s128) * (1 + 2.0 ** -18) + \
        2 * e * want.abs()
    assert ((b.q.cpu().double() * s128 - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype,gain_dtype", [(BF, BF), (F16, F16), (BF, F32)])
@pytest.mark.parametrize("with_ds", [False, True])
@pytest.mark.parametrize("n,cols", [(1, 1), (3, 7), (5, 129), (300, 64), (9, 1408), (700, 520),
                                    (4, 2049), (3, 5000), (3, 9001), (2, 16384), (3, 20000)])
def test_backward(ctx, n, cols, with_ds, dtype, gain_dtype):
    s, hs = rows_of(n, cols, dtype, cols, spread=2.0)
    dy, hy = rows_of(n, cols, dtype, cols + 1, spread=0.1)
    ds, hd = rows_of(n, cols, dtype, cols + 2, spread=0.1)
    gain, hg = gain_of(cols, gain_dtype, cols + 3)
    dx, dgain = ctx.rms_norm_backward(dy, s, gain, EPS, ds=ds if with_ds else None)
    hs, hy, hd, hg = (t.double() for t in (hs, hy, hd, hg))
    if not with_ds:
        hd = torch.zeros_like(hd)
    r = norm(hs, hg, EPS)[1]
    u, du = hs * r, hy * hg
    mean = (du * u).mean(dim=1, keepdim=True)
    want = hd + r * (du - u * mean)
    # each term's own error and the mean's, whose sum of magnitudes is the larger
    size = hd.abs() + r * (du.abs() + u.abs() * (du * u).abs().mean(dim=1, keepdim=True))
    e = 3 * f32_error(cols)
    tol = HALF[dtype] * want.abs() + (1 + HALF[dtype]) * e * size + TINY[dtype]
    assert ((dx.cpu().double() - want).abs() <= tol).all()
    assert dgain.dtype == gain_dtype
    want, size = (hy * u).sum(dim=0), (hy * u).abs().sum(dim=0)
    # a row's own error, and fewer additions than rows + 32
    tol = (HALF.get(gain_dtype, 2.0 ** -24) * want.abs() + (e + (n + 32) * 2.0 ** -24) * size +
           TINY.get(gain_dtype, 0.0))
    assert ((dgain.cpu().double() - want).abs() <= tol).all()


def test_backward_against_differences(T, ctx):
    """The gradients of a loss against central differences of the formula in 64 bits."""
    n, cols = 4, 200
    x, hx = rows_of(n, cols, F16, 1)
    r, hr = rows_of(n, cols, F16, 2)
    gain, hg = gain_of(cols, F32, 3)
    a, b = torch.randn(n, cols, dtype=torch.float64), torch.randn(n, cols, dtype=torch.float64)
    a, b = a.half().double(), b.half().double()
    x.requires_grad_(), r.requires_grad_(), gain.requires_grad_()
    y, total = T.rms_norm(ctx, x, gain, EPS, residual=r)
    torch.autograd.backward([y, total], [a.half().cuda(), b.half().cuda()])
    assert torch.equal(x.grad, r.grad)

    def loss(s, g):
        return float((norm(s, g, EPS)[0] * a).sum() + (s * b).sum())

    s, g = hx.double() + hr.double(), hg.double()
    h = 1e-5
    for i, j in [(0, 0), (1, 17), (2, 128), (3, 199)]:
        d = torch.zeros(n, cols, dtype=torch.float64)
        d[i, j] = h
        slope = (loss(s + d, g) - loss(s - d, g)) / (2 * h)
        # the stored sum is rounded to 16 bits and so is the gradient: half a step of each,
        # the former through slopes of about the gradient's size
        assert abs(slope - float(x.grad[i, j])) <= 4 * 2.0 ** -11 * (abs(slope) + 1.0)
        e = torch.zeros(cols, dtype=torch.float64)
        e[j] = h
        slope = (loss(s, g + e) - loss(s, g - e)) / (2 * h)
        assert abs(slope - float(gain.grad[j])) <= 4 * 2.0 ** -11 * (abs(slope) + 1.0)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("cols", [200, 4096, 20000])
def test_rows_beyond_binary32s_squares(ctx, dtype, cols):
    """Rows whose squares overflow or vanish, beside ordinary ones, an infinite and a NaN one."""
    x, _ = rows_of(7, cols, dtype, 5)
    if dtype == BF:
        x[1] *= 1e25
        x[2] *= 1e-30
    x[3] = 0
    x[4, 3] = float("inf")
    x[5, 7] = float("nan")
    x[6] = torch.finfo(dtype).max
    host = x.cpu()
    gain, hg = gain_of(cols, dtype, 6)
    for eps in (EPS, 1e-30):
        want, r = norm(host, hg, eps)
        y = ctx.rms_norm(x, gain, eps).cpu().double()
        e = f32_error(cols)
        for t in (0, 1, 2, 3, 6):
            tol = want[t].abs() * (HALF[dtype] * (1 + 2 * e) + e) + TINY[dtype]
            assert ((y[t] - want[t]).abs() <= tol).all(), (eps, t)
        assert torch.isnan(y[5]).all()
        b = ctx.rms_norm(x, gain, eps, blocks=True)
        assert torch.isnan(b.scale[5]).all() and torch.isnan(b.q[5].float()).all()
        assert (b.q[3].float() == 0).all()
        # gradients of the rows with finite values
        dy, hy = rows_of(7, cols, dtype, 8, spread=0.1)
        dx, _ = ctx.rms_norm_backward(dy, x, gain, eps)
        u, du = host.double() * r, hy.double() * hg.double()
        ref = r * (du - u * (du * u).mean(dim=1, keepdim=True))
        size = r * (du.abs() + u.abs() * (du * u).abs().mean(dim=1, keepdim=True))
        for t in (0, 1, 2, 3, 6):
            inside = ref[t].abs() < torch.finfo(dtype).max * 0.99
            tol = HALF[dtype] * ref[t].abs() + 4 * e * size[t] + TINY[dtype]
            off = (dx[t].cpu().double() - ref[t]).abs()
            assert (off[inside] <= tol[inside]).all(), (eps, t)


@pytest.mark.parametrize("cols", [200, 3000, 20000])
def test_in_place(ctx, cols):
    """The sum over the residual, the result over x, and both the other way round."""
    gain, _ = gain_of(cols, BF, 1)
    x, _ = rows_of(5, cols, BF, 2)
    r, _ = rows_of(5, cols, BF, 3)
    y, total = ctx.rms_norm(x, gain, EPS, residual=r)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        y2, t2 = ctx.rms_norm(a, gain, EPS, residual=b, out=b if swap else a,
                              sum_out=a if swap else b)
        assert torch.equal(y2, y) and torch.equal(t2, total)
    a = x.clone()
    assert torch.equal(ctx.rms_norm(a, gain, EPS, out=a), ctx.rms_norm(x, gain, EPS))


@pytest.mark.parametrize("cols", [1, 130, 1000, 3001])
def test_rows_of_any_pitch_and_nothing_behind_them(ctx, cols):
    gain, hg = gain_of(cols, BF, 1)
    for pitch, at in [(cols, 0), (cols + 1, 1), (cols + 9, 3), (cols + 16, 8)]:
        x, hx = rows_of(4, cols, BF, 2, pitch=pitch, at=at)
        r, hr = rows_of(4, cols, BF, 3, pitch=pitch + 1, at=at)
        out = torch.full((4 * (pitch + 2) + 9,), 9.0, dtype=BF, device="cuda")
        tot = out.clone()

        def inside(t):
            return t[at:].as_strided((4, cols), (pitch + 2, 1))

        y, total = ctx.rms_norm(x, gain, EPS, residual=r, out=inside(out), sum_out=inside(tot))
        want, _ = ctx.rms_norm(hx.cuda(), gain, EPS, residual=hr.cuda())
        assert torch.equal(y, want) and torch.equal(total.cpu(), (hx.float() + hr.float()).to(BF))
        for t in (out, tot):
            inside(t).fill_(9.0)
            assert (t == 9).all()


def test_the_gains_gradient_without_rows_and_what_is_not_wanted(ctx):
    gain, _ = gain_of(300, BF, 1)
    none = torch.zeros(0, 300, dtype=BF, device="cuda")
    assert ctx.rms_norm(none, gain).shape == (0, 300)
    b = ctx.rms_norm(none, gain, blocks=True)
    assert b.q.shape == (0, 300) and b.scale.shape == (0, 3)
    dx, dgain = ctx.rms_norm_backward(none, none, gain)
    assert dx.shape == (0, 300) and (dgain == 0).all()
    x, _ = rows_of(5, 300, BF, 2)
    both = ctx.rms_norm_backward(x, x, gain)
    dx, no = ctx.rms_norm_backward(x, x, gain, want_dgain=False)
    assert no is None and torch.equal(dx, both[0])
    no, dgain = ctx.rms_norm_backward(x, x, gain, want_dx=False)
    assert no is None and torch.equal(dgain, both[1])


def test_gradients_of_one_result_only(T, ctx):
    gain, _ = gain_of(300, BF, 1)
    x, _ = rows_of(6, 300, BF, 2)
    r, _ = rows_of(6, 300, BF, 3)
    g, _ = rows_of(6, 300, BF, 4)
    for use in ("y", "total"):
        a, b, c = x.clone().requires_grad_(), r.clone().requires_grad_(), gain.clone().requires_grad_()
        y, total = T.rms_norm(ctx, a.reshape(2, 3, 300), c, EPS, residual=b.reshape(2, 3, 300))
        (y if use == "y" else total).backward(g.reshape(2, 3, 300))
        if use == "total":
            assert torch.equal(a.grad, g) and torch.equal(b.grad, g) and (c.grad == 0).all()
        else:
            dx, dgain = ctx.rms_norm_backward(g, total.detach().reshape(6, 300), gain, EPS)
            assert torch.equal(a.grad, dx) and torch.equal(b.grad, dx)
            assert torch.equal(c.grad, dgain)
    # a frozen gain, no residual
    a = x.clone().requires_grad_()
    T.rms_norm(ctx, a, gain, EPS).backward(g)
    assert torch.equal(a.grad, ctx.rms_norm_backward(g, x, gain, EPS)[0])


def test_a_layers_step_forward_and_backward(T, ctx):
    """Norm, product, norm, product by expert, with the gradients, as a layer uses them."""
    from block_reference import from_blocks, to_blocks
    g = torch.Generator().manual_seed(9)
    dim, wide, n = 256, 384, 50
    w1 = ctx.block_quantize_weight((torch.randn(wide, dim, generator=g) * 0.06).to(BF).cuda())
    w2 = ctx.block_quantize_weight((torch.randn(3, dim, wide, generator=g) * 0.05).to(BF).cuda())
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32).cuda()
    x, _ = rows_of(n, dim, BF, 1)
    res, _ = rows_of(n, dim, BF, 2)
    gain, _ = gain_of(dim, BF, 3)
    x.requires_grad_(), res.requires_grad_(), gain.requires_grad_()
    y, s = T.rms_norm(ctx, x, gain, EPS, residual=res)
    h = T.block_linear(ctx, y, w1)
    out = T.block_grouped_linear(ctx, torch.relu(h), w2, off) + s
    out.float().square().sum().backward()

    # the same in 64 bits from the values that the 8-bit forms stand for, rounding passed through
    def through(v):
        q, sc = to_blocks(v.detach().to(BF).float())
        return v + (from_blocks(q, sc) - v).detach()

    hx, hr, hg = (t.detach().cpu().double().requires_grad_() for t in (x, res, gain))
    sum_ = hx + hr
    yy = norm(sum_, hg, EPS)[0]
    hh = through(yy) @ w1.dequantize().cpu().double().t()
    act = through(torch.relu(hh))
    e2 = w2.dequantize().cpu().double()
    oo = torch.cat([act[:20] @ e2[0].t(), act[20:] @ e2[2].t()]) + sum_
    oo.square().sum().backward()
    # 16-bit and 8-bit roundings of values and gradients all through the chain: e4m3's 2^-4 at
    # most on each of four operands, averaged over contractions of 256 and more
    assert float((out.detach().cpu().double() - oo.detach()).norm() / oo.detach().norm()) < 0.02
    for got, want in ((x.grad, hx.grad), (res.grad, hr.grad), (gain.grad, hg.grad)):
        assert float((got.cpu().double() - want).norm() / want.norm()) < 0.06
    # and the 8-bit output of the norm is the product's operand
    b, _ = ctx.rms_norm(x.detach(), gain.detach(), EPS, residual=res.detach(), blocks=True)
    hb = ctx.block_linear(b, w1)
    assert float((hb.double() - h.detach().double()).norm() / h.detach().double().norm()) < 0.05


def test_backward_captured_and_replayed(T):
    gain, _ = gain_of(1000, BF, 1)
    s, _ = rows_of(300, 1000, BF, 2)
    dy, _ = rows_of(300, 1000, BF, 3)
    with T.Context(0) as c, T.Context(0) as other:
        c.rms_norm_backward(dy, s, gain)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = c.rms_norm_backward(dy, s, gain)
        for seed in range(4):
            new, _ = rows_of(300, 1000, BF, 10 + seed)
            s.copy_(new)
            want = other.rms_norm_backward(dy, s, gain)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(c.rms_norm_backward(dy, s, gain)[1], want[1])
        torch.cuda.synchronize()
        del graph


def test_refusals(T, ctx):
    x, _ = rows_of(4, 256, BF, 1)
    gain, _ = gain_of(256, BF, 2)
    for call in [lambda: ctx.rms_norm(x, gain[:255]), lambda: ctx.rms_norm(x, gain.half()),
                 lambda: ctx.rms_norm(x, gain.double()), lambda: ctx.rms_norm(x.float(), gain),
                 lambda: ctx.rms_norm(x, gain, residual=x[:3]),
                 lambda: ctx.rms_norm(x, gain, residual=x.half()),
                 lambda: ctx.rms_norm(x, gain, sum_out=x),
                 lambda: ctx.rms_norm(x, gain, blocks=True, out=x),
                 lambda: ctx.rms_norm(x[0], gain), lambda: ctx.rms_norm(x, gain.cpu()),
                 lambda: ctx.rms_norm_backward(x[:3], x, gain),
                 lambda: ctx.rms_norm_backward(x, x, gain, ds=x.half())]:
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(4, 600, dtype=BF, device="cuda")
    for call in [lambda: ctx.rms_norm(x, gain, eps=-1.0),
                 lambda: ctx.rms_norm(x, gain, eps=float("nan")),
                 lambda: ctx.rms_norm(x, gain, eps=float("inf")),
                 lambda: ctx.rms_norm(wide[:, :256], gain, out=wide[:, 100:356]),
                 lambda: ctx.rms_norm(x, gain, residual=wide[:, :256], sum_out=wide[:, 8:264]),
                 lambda: ctx.rms_norm(x, gain, residual=x, out=wide[:, :256], sum_out=wide[:, :256]),
                 lambda: ctx.rms_norm_backward(x, x, gain, eps=-1.0)]:
        with pytest.raises(T.Exl3Error) as e:
            call()
        assert e.value.code == T.EXL3_EINVAL
