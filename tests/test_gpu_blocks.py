"""Operators in 8-bit blocks on the GPU: writing blocks, products, products by expert, against the
reference in 64 bits (block_reference.py)."""
import pytest
import torch

from block_reference import E4M3, HALF, TINY, blocks, from_blocks, product, rows_of, to_blocks

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    with T.Context(0) as c:
        yield c


def same_codes(got, want):
    """Bit for bit, where a NaN is any NaN."""
    g, w = got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)
    nan = (w & 0x7F) == 0x7F
    return torch.equal((g & 0x7F) == 0x7F, nan) and torch.equal(g[~nan], w[~nan])


def same_scales(got, want):
    return torch.equal(got.cpu().nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


def matrix(rows, cols, seed, groups=None):
    """(codes, scales) of a matrix with a few empty rows, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(groups or 1):
        w = torch.randn(rows, cols, generator=g) * 0.02
        w = w * torch.exp(0.4 * torch.randn(rows, 1, generator=g))
        w = torch.where(torch.rand(rows, 1, generator=g) < 0.03, 0.0, w)
        out.append(to_blocks(w, 128))
    if groups is None:
        return out[0]
    return torch.stack([q.view(torch.uint8) for q, _ in out]).view(E4M3), \
        torch.stack([s for _, s in out])


def UNIT(k):
    """What the matrix units and the sums of their results lose at most of the magnitudes' sum."""
    return 7 * 2.0 ** -13 + (19 + blocks(k)) * 2.0 ** -24


def check_product(y, x, w, dtype, k):
    """y against x w^T in 64 bits.  The matrix units align eight products of neighbouring k's to the
    largest of them and keep 13 bits below its leading one (of 2^16 and 2^s at two of eight
    neighbouring k's the sum is exact down to s = 3 and 2^16 from s = 2 on; products of different
    eights meet in binary32): the other seven lose less than 2^-13 of the largest each, together
    less than 7 * 2^-13 of the eight's magnitudes.  Then at most 16 + blocks + 3 roundings of 2^-24
    on any product's way, and one to the result's type."""
    want, size = product(x, w)
    y = y.cpu().double()
    tol = HALF[dtype] * want.abs() + 1.01 * UNIT(k) * size + TINY[dtype]
    bad = (y - want).abs() > tol
    assert not bad.any(), "%d of %d off, worst %g of the tolerance" % (
        int(bad.sum()), bad.numel(), float(((y - want).abs() / tol).max()))


SIZES = [(1, 1), (1, 128), (2, 127), (3, 129), (5, 257), (33, 1000), (128, 1408), (7, 5000)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("n,cols", SIZES)
def test_rows_as_blocks_bit_for_bit(ctx, n, cols, dtype):
    x, host = rows_of(n, cols, dtype, 11 * n + cols)
    got = ctx.block_quantize(x)
    q, scale = to_blocks(host.float())
    assert got.q.shape == (n, cols) and got.scale.shape == (n, blocks(cols))
    assert same_codes(got.q, q) and same_scales(got.scale, scale)
    assert torch.equal(got.dequantize().cpu(),
                       q.float() * scale.repeat_interleave(128, 1)[:, :cols])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_blocks_of_extreme_values(ctx, dtype):
    """Zero blocks, the smallest and largest values, exact ties, infinities and NaN."""
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    rows = torch.zeros(12, 300)
    rows[1, 5] = small * 2 ** -5
    rows[2, :] = big
    rows[3, ::2], rows[3, 1::2] = big, -big / 2
    rows[4, :] = torch.arange(300) - 150.0
    rows[5, :] = (torch.arange(300) % 128 + 1) / 128.0         # 0.75 of the largest is a tie
    rows[6, 130] = float("inf")
    rows[7, 299] = float("-inf")
    rows[8, 0] = float("nan")
    rows[9, :] = small
    rows[10, :] = 448.0
    rows[10, 1::2] = 7.0 * 2.0 ** -9                           # codes between the subnormal ones
    rows[11, :] = -0.0
    host = rows.to(dtype)
    got = ctx.block_quantize(host.cuda())
    q, scale = to_blocks(host.float())
    assert same_scales(got.scale, scale) and same_codes(got.q, q)


@pytest.mark.parametrize("dtype", [torch.float32, BF, F16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 130), (300, 1000), (257, 384)])
def test_a_matrix_as_blocks_bit_for_bit(ctx, rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    w = (torch.randn(rows, cols, generator=g) * 0.02).to(dtype)
    if rows > 2:
        w[rows // 2] = 0
    got = ctx.block_quantize_weight(w.cuda())
    q, scale = to_blocks(w.float(), 128)
    assert same_codes(got.q, q) and same_scales(got.scale, scale)
    # the zeros behind the last column belong to the storage
    wide = got.q.as_strided((rows, 128 * blocks(cols)), (128 * blocks(cols), 1))
    assert (wide[:, cols:].view(torch.uint8) == 0).all()


def test_matrices_of_any_pitch_and_groups(ctx):
    g = torch.Generator().manual_seed(5)
    w = torch.randn(3, 140, 200, generator=g).to(BF)
    w[1, 130, 3] = float("nan")
    got = ctx.block_quantize_weight(w.cuda())
    for e in range(3):
        q, scale = to_blocks(w[e].float(), 128)
        assert same_codes(got.q[e], q) and same_scales(got.scale[e], scale)
    part = ctx.block_quantize_weight(w.cuda()[0, 3:, 7:190])
    q, scale = to_blocks(w[0, 3:, 7:190].float(), 128)
    assert same_codes(part.q, q) and same_scales(part.scale, scale)


PRODUCTS = [(1, 1, 1), (1, 128, 128), (2, 130, 100), (3, 16, 257), (16, 256, 2048),
            (17, 300, 129), (33, 1000, 400), (64, 257, 1000), (100, 64, 5000), (130, 129, 384),
            (200, 1408, 512), (257, 513, 640), (600, 384, 256)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("form", ["rows", "blocks", "transposed"])
@pytest.mark.parametrize("n,rows,cols", PRODUCTS)
def test_products(T, ctx, n, rows, cols, form, dtype):
    q, scale = matrix(rows, cols, 3 * n + rows + cols)
    w = T.BlockWeight(q.cuda(), scale.cuda())
    back = form == "transposed"
    k = rows if back else cols
    x, host = rows_of(n, k, dtype, n + 7 * rows + cols)
    xq, xs = to_blocks(host.float())
    if form == "blocks":
        y = ctx.block_linear(T.BlockRows(xq.cuda(), xs.cuda()), w, dtype=dtype)
    else:
        y = ctx.block_linear(x, w, transpose=back)
    assert y.dtype == dtype and y.shape == (n, cols if back else rows)
    dense = from_blocks(q, scale, 128)
    check_product(y, from_blocks(xq, xs), dense.t() if back else dense, dtype, k)


GROUPS = [
    (4, 300, 260, [0, 3, 3, 40, 41]),                  # an empty group, one row, 37
    (3, 129, 384, [2, 2, 50, 60]),                     # rows before the first and after the last
    (5, 128, 640, [0, 0, 0, 0, 0, 0]),                 # no rows at all in groups
    (2, 257, 130, [0, 200, 333]),
    (8, 64, 1000, [1, 130, 131, 131, 260, 300, 301, 310, 320]),
    (70, 130, 256, list(range(71))),                   # more groups than a wave has lanes
]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("form", ["rows", "blocks", "transposed"])
@pytest.mark.parametrize("E,rows,cols,offsets", GROUPS)
def test_products_by_group(T, ctx, E, rows, cols, offsets, form, dtype):
    n = offsets[-1] + 5
    q, scale = matrix(rows, cols, E + rows + cols, groups=E)
    w = T.BlockWeight(q.cuda(), scale.cuda())
    back = form == "transposed"
    k, m = (rows, cols) if back else (cols, rows)
    x, host = rows_of(n, k, dtype, E + n)
    xq, xs = to_blocks(host.float())
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    out = torch.full((n + 2, m + 3), 5.0, dtype=dtype, device="cuda")
    given = T.BlockRows(xq.cuda(), xs.cuda()) if form == "blocks" else x
    y = ctx.block_grouped_linear(given, w, off, transpose=back, out=out[:n, :m])
    assert (out[n:] == 5).all() and (out[:, m:] == 5).all()
    rowsx = from_blocks(xq, xs)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        dense = from_blocks(q[e], scale[e], 128)
        if b > a:
            check_product(y[a:b], rowsx[a:b], dense.t() if back else dense, dtype, k)
    assert (y[:offsets[0]] == 0).all() and (y[offsets[-1]:] == 0).all()


@pytest.mark.parametrize("n", [1, 20, 150])
def test_rows_of_any_pitch_and_alignment(T, ctx, n):
    q, scale = matrix(200, 300, 21)
    w = T.BlockWeight(q.cuda(), scale.cuda())
    for pitch, at in [(300, 0), (301, 1), (309, 3), (320, 8)]:
        x, host = rows_of(n, 300, BF, 31, pitch=pitch, at=at)
        out = torch.full((1 + n * 213 + 50,), 9.0, dtype=BF, device="cuda")
        y = out[1:].as_strided((n, 200), (213, 1))
        ctx.block_linear(x, w, out=y)
        xq, xs = to_blocks(host.float())
        check_product(y, from_blocks(xq, xs), from_blocks(q, scale, 128), BF, 300)
        rest = out.clone()
        rest[1:].as_strided((n, 200), (213, 1)).fill_(9.0)
        assert (rest == 9).all()


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n", [1, 12, 40, 200])
def test_a_bad_row_or_channel_stays_its_own(T, ctx, n, back):
    q, scale = matrix(256, 384, 41)
    k, m = (256, 384) if back else (384, 256)
    codes = q.view(torch.uint8).clone()
    if back:
        codes[7, 100] = 0x7F
    else:
        codes[100, 7] = 0x7F
    w = T.BlockWeight(codes.view(E4M3).cuda(), scale.cuda())
    x, host = rows_of(n, k, BF, 43)
    clean = ctx.block_linear(x, T.BlockWeight(q.cuda(), scale.cuda()), transpose=back)
    bad = min(n - 1, 5)
    x[bad, 200] = float("nan") if n % 8 else float("inf")
    y = ctx.block_linear(x, w, transpose=back)
    assert torch.isnan(y[bad]).all() and torch.isnan(y[:, 100]).all()
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[100] = False
    rest = torch.arange(n, device="cuda") != bad
    assert torch.equal(y[rest][:, keep], clean[rest][:, keep])


def test_a_weight_whose_last_block_has_few_rows_and_a_nan_in_it(T, ctx):
    """Transposed, the rows past the last are read as repeats of it: nothing of them shows."""
    q, scale = matrix(130, 128, 45)
    w = T.BlockWeight(q.cuda(), scale.cuda())
    x, host = rows_of(9, 130, BF, 46)
    xq, xs = to_blocks(host.float())
    y = ctx.block_linear(x, w, transpose=True)
    check_product(y, from_blocks(xq, xs), from_blocks(q, scale, 128).t(), BF, 130)


def test_scales_of_the_blocks_reach_the_results(T, ctx):
    """Every scale of x and of W another power of two: no scale stands for another."""
    R, C, n = 400, 520, 37
    g = torch.Generator().manual_seed(3)
    q = torch.randint(0, 2, (R, C), generator=g).float().mul(2).sub(1).to(E4M3)
    s = torch.exp2(torch.randint(-6, 6, (blocks(R), blocks(C)), generator=g).float())
    xq = torch.randint(0, 2, (n, C), generator=g).float().mul(2).sub(1).to(E4M3)
    xs = torch.exp2(torch.randint(-6, 6, (n, blocks(C)), generator=g).float())
    y = ctx.block_linear(T.BlockRows(xq.cuda(), xs.cuda()), T.BlockWeight(q.cuda(), s.cuda()))
    check_product(y, from_blocks(xq, xs), from_blocks(q, s, 128), BF, C)


def test_holders_keep_whole_blocks_and_copy_others(T):
    q, s = matrix(130, 256, 51)
    q, s = q.cuda(), s.cuda()
    assert T.BlockWeight(q, s).q.data_ptr() == q.data_ptr()
    xs = torch.rand(2, 6, device="cuda").t()
    rows = T.BlockRows(q[:6], xs)
    assert rows.q.data_ptr() == q.data_ptr() and rows.scale.data_ptr() == xs.data_ptr()
    odd, so = matrix(6, 130, 52)
    rows = T.BlockRows(odd.cuda(), torch.rand(6, 2, device="cuda"))
    assert rows.q.stride(0) == 256 and rows.scale.stride(0) == 1
    assert torch.equal(rows.q.cpu().view(torch.uint8), odd.view(torch.uint8))
    part = T.BlockRows(q[3:4, :128], xs[:1, :1])
    assert part.n == 1 and part.cols == 128


def test_no_rows(T, ctx):
    q, s = matrix(130, 256, 53)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x = torch.zeros(0, 256, dtype=BF, device="cuda")
    assert ctx.block_linear(x, w).shape == (0, 130)
    assert ctx.block_linear(ctx.block_quantize(x), w).shape == (0, 130)
    assert ctx.block_linear(torch.zeros(0, 130, dtype=BF, device="cuda"), w,
                            transpose=True).shape == (0, 256)


def test_a_coded_weight_as_blocks(T, ctx):
    from product_reference import dense, random_weight
    from test_gpu_products import on_gpu
    for K, had, groups in [(2, 128, None), (3, 64, None)]:
        host = random_weight(256, 384, K, had, 61)
        w = ctx.block_weight(on_gpu(T, host))
        want = torch.from_numpy(dense(host))
        # the decoded weight's own binary32 roundings, then half a step of e4m3 of the block
        got = w.dequantize().cpu().double()
        scale = w.scale.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scale) * (1 + 2.0 ** -12) + \
            64 * 2.0 ** -24 * want.abs().max()
        assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("n", [3, 300])
def test_the_same_results_every_time(T, ctx, n):
    q, s = matrix(1000, 2048, 71)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(n, 2048, BF, 72)
    first = ctx.block_linear(x, w)
    for _ in range(5):
        assert torch.equal(ctx.block_linear(x, w), first)


@pytest.mark.parametrize("n", [2, 40, 300])
def test_captured_and_replayed_with_eager_work_between(T, n):
    q, s = matrix(260, 384, 81)
    w = T.BlockWeight(q.cuda(), s.cuda())
    with T.Context(0) as c, T.Context(0) as other:
        x, _ = rows_of(n, 384, BF, 82)
        gain = torch.ones(384, dtype=BF, device="cuda")

        def step(c):
            y, total = c.rms_norm(x, gain, residual=x, blocks=True)
            return c.block_linear(y, w), c.block_linear(x, w), total

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(c)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(c)
        for seed in range(4):
            xn, _ = rows_of(n, 384, BF, 90 + seed)
            x.copy_(xn)
            want = step(other)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            assert torch.equal(step(c)[1], want[1])
        torch.cuda.synchronize()
        del graph


def test_on_another_stream_than_the_tensors(T, ctx):
    q, s = matrix(512, 1024, 91)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(64, 1024, BF, 92)
    want = ctx.block_linear(x, w)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(1000000)
        y = ctx.block_linear(x, w)
    stream.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(ctx.block_linear(x, w), want)


def test_timing_has_one_record_a_call(T):
    q, s = matrix(256, 256, 95)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(8, 256, BF, 96)
    with T.Context(0) as c:
        c.set_timing(True)
        c.block_linear(x, w)
        c.block_linear(c.block_quantize(x), w)
        ms, launches, tiles = c.read_timing("block")
        assert launches == 2 and tiles == 8 and ms > 0
        assert c.read_timing("norm")[1] == 1


def test_refusals(T, ctx):
    q, s = matrix(256, 384, 97)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(4, 384, BF, 98)
    for call in [lambda: ctx.block_linear(x[:, :383], w),
                 lambda: ctx.block_linear(x.float(), w),
                 lambda: ctx.block_linear(x.cpu(), w),
                 lambda: ctx.block_linear(x, w, dtype=F16),
                 lambda: ctx.block_linear(x, w, transpose=True),
                 lambda: ctx.block_linear(ctx.block_quantize(x), w, dtype=torch.float32),
                 lambda: ctx.block_linear(x, w, out=torch.empty(4, 255, dtype=BF, device="cuda")),
                 lambda: ctx.block_grouped_linear(x, w, torch.zeros(3, dtype=torch.int32).cuda()),
                 lambda: T.BlockRows(q.cuda(), s.cuda()),
                 lambda: T.BlockRows(q.cuda().float(), s.cuda()),
                 lambda: T.BlockWeight(q.cuda(), s.cuda().t()),
                 lambda: T.BlockWeight(q.cuda(), s),
                 lambda: T.BlockWeight(q.cuda(), s.cuda().double()),
                 lambda: ctx.block_quantize_weight(q.cuda().double()),
                 lambda: ctx.block_quantize(x.float())]:
        with pytest.raises(ValueError):
            call()
    both = T.BlockWeight(torch.stack([q.view(torch.uint8)] * 2).view(E4M3).cuda(),
                         torch.stack([s, s]).cuda())
    with pytest.raises(ValueError):
        ctx.block_linear(x, both)
    square, ss = matrix(384, 384, 99)
    with pytest.raises(T.Exl3Error) as e:
        ctx.block_linear(x, T.BlockWeight(square.cuda(), ss.cuda()), out=x)
    assert e.value.code == T.EXL3_EINVAL


def test_the_c_entries_refuse_what_the_binding_never_passes(T, ctx):
    import ctypes
    q, s = matrix(256, 384, 97)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(4, 384, BF, 98)
    y = torch.zeros(4, 256, dtype=BF, device="cuda")
    rows = ctx.block_quantize(x)
    lib, h = ctx.lib, ctx.handle
    cw, cb = type(w._c), type(rows._c)

    def linear(weight, xp, blocks_, n=4, dtype=T.EXL3_BF16):
        return lib.exl3_block_linear(h, weight, 0, xp, 384, blocks_, n, dtype, y.data_ptr(), 256)

    def weight(**kw):
        f = dict(q=w._c.q, scale=w._c.scale, groups=1, rows=256, cols=384, ldq=384)
        f.update(kw)
        return ctypes.byref(cw(f["q"], f["scale"], f["groups"], f["rows"], f["cols"], f["ldq"]))

    def given(**kw):
        f = dict(q=rows._c.q, scale=rows._c.scale, ldq=384, lds=4)
        f.update(kw)
        return ctypes.byref(cb(f["q"], f["scale"], f["ldq"], f["lds"]))

    for bad in [linear(None, x.data_ptr(), None), linear(weight(q=None), x.data_ptr(), None),
                linear(weight(scale=None), x.data_ptr(), None),
                linear(weight(ldq=385), x.data_ptr(), None),
                linear(weight(ldq=256), x.data_ptr(), None),
                linear(weight(q=w._c.q + 8), x.data_ptr(), None),
                linear(weight(rows=0), x.data_ptr(), None),
                linear(weight(rows=1 << 21), x.data_ptr(), None),
                linear(weight(groups=0), x.data_ptr(), None),
                linear(weight(groups=2), x.data_ptr(), None),
                linear(weight(), None, None), linear(weight(), x.data_ptr(), given()),
                linear(weight(), None, given(ldq=400)), linear(weight(), None, given(lds=3)),
                linear(weight(), None, given(q=rows._c.q + 4)),
                linear(weight(), None, given(scale=None)),
                linear(weight(), x.data_ptr(), None, n=-1),
                linear(weight(), x.data_ptr(), None, n=(1 << 24) + 1),
                linear(weight(), x.data_ptr(), None, dtype=T.EXL3_F32),
                linear(weight(), x.data_ptr(), None, n=1 << 20),
                lib.exl3_block_grouped_linear(h, weight(), None, 0, x.data_ptr(), 384, None, 4,
                                              T.EXL3_BF16, y.data_ptr(), 256),
                lib.exl3_block_quantize(h, x.data_ptr(), 384, 4, 384, T.EXL3_BF16,
                                        given(q=x.data_ptr())),
                lib.exl3_block_quantize(h, x.data_ptr(), 384, 4, 0, T.EXL3_BF16, given()),
                lib.exl3_block_quantize_weight(h, x.data_ptr(), 383, 4, 384, T.EXL3_BF16, w._c.q,
                                               384, w._c.scale),
                lib.exl3_block_quantize_weight(h, x.data_ptr(), 384, 4, 384, 7, w._c.q, 384,
                                               w._c.scale),
                lib.exl3_block_quantize_weight(h, x.data_ptr(), 384, 4, 384, T.EXL3_BF16,
                                               x.data_ptr(), 384, w._c.scale)]:
        assert bad == T.EXL3_EINVAL
    assert linear(weight(), x.data_ptr(), None) == T.EXL3_OK
    torch.cuda.synchronize()


def test_differentiable_products(T, ctx):
    """The gradient is that of the formula; and, at values that e4m3 holds exactly, the difference
    of two forward passes is its product with their distance."""
    q, s = matrix(300, 256, 101)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, host = rows_of(24, 256, BF, 102)
    x = x.reshape(2, 12, 256).requires_grad_()
    y = T.block_linear(ctx, x, w)
    dy, dhost = rows_of(24, 300, BF, 103)
    y.backward(dy.reshape(2, 12, 300))
    dq, ds = to_blocks(dhost.float())
    dense = from_blocks(q, s, 128)
    check_product(x.grad.reshape(24, 256), from_blocks(dq, ds), dense.t(), BF, 300)
    g = torch.Generator().manual_seed(5)
    a = torch.randint(-8, 9, (24, 256), generator=g).float()
    a[:, ::128] = 14.0                                     # 14 / 448 is a power of two
    b = a.clone()
    b[:, 5] += 1.0                                         # still whole numbers below 16
    ya = ctx.block_linear(a.to(F16).cuda(), w).double().cpu()
    yb = ctx.block_linear(b.to(F16).cuda(), w).double().cpu()
    _, size = product(a.abs() + 1, dense)
    tol = 2.0 ** -11 * (ya.abs() + yb.abs()) + 2.1 * UNIT(256) * size
    assert ((yb - ya - dense[:, 5]).abs() <= tol).all()
    off = torch.tensor([0, 10, 24], dtype=torch.int32).cuda()
    two = T.BlockWeight(torch.stack([q.view(torch.uint8)] * 2).view(E4M3).cuda(),
                        torch.stack([s, 2 * s]).cuda())
    xg = x.detach().reshape(24, 256).requires_grad_()
    T.block_grouped_linear(ctx, xg, two, off).backward(dy)
    # (against the formula: a single matrix and groups may add a contraction's blocks in another
    # order, each within the same bound)
    ref = from_blocks(dq, ds)
    check_product(xg.grad[:10], ref[:10], dense.t(), BF, 300)
    check_product(xg.grad[10:], ref[10:], 2 * dense.t(), BF, 300)


LONG = [(3, 40, 9000), (20, 40, 20000), (40, 70, 20000), (200, 260, 17000), (300, 1100, 8200)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n,m,k", LONG)
def test_long_contractions(T, ctx, n, m, k, back):
    """More blocks than a wave has lanes, in every tile."""
    rows, cols = (k, m) if back else (m, k)
    q, scale = matrix(rows, cols, n + m + k)
    x, host = rows_of(n, k, BF, n + k)
    xq, xs = to_blocks(host.float())
    y = ctx.block_linear(x, T.BlockWeight(q.cuda(), scale.cuda()), transpose=back)
    dense = from_blocks(q, scale, 128)
    check_product(y, from_blocks(xq, xs), dense.t() if back else dense, BF, k)


# sizes at which each of the tiles is chosen (one matrix), by rows and result columns
TILES = [(4096, 4096, 1030), (1500, 4096, 1300), (3840, 2176, 900), (1000, 4096, 1100),
         (500, 4096, 1200), (150, 4096, 1390), (100, 4096, 2000), (60, 4096, 1500),
         (1800, 4100, 128)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n,m,k", TILES)
def test_every_tile(T, ctx, n, m, k, back):
    rows, cols = (k, m) if back else (m, k)
    q, scale = matrix(rows, cols, n + m)
    x, host = rows_of(n, k, BF, n + k)
    xq, xs = to_blocks(host.float())
    y = ctx.block_linear(x, T.BlockWeight(q.cuda(), scale.cuda()), transpose=back)
    dense = from_blocks(q, scale, 128)
    dense = dense.t() if back else dense
    # a sample of the rows, the first and the last tiles among them
    at = torch.cat([torch.arange(0, n, 37), torch.arange(max(0, n - 40), n)])
    check_product(y[at.cuda()], from_blocks(xq, xs)[at], dense, BF, k)
    assert torch.equal(y, ctx.block_linear(ctx.block_quantize(x), T.BlockWeight(q.cuda(), scale.cuda()),
                                           transpose=back))


@pytest.mark.parametrize("back", [False, True])
def test_many_groups_of_many_rows(T, ctx, back):
    """Tiles of experts' rows: empty groups, groups of one row and of several tiles."""
    sizes = [0, 1, 700, 0, 129, 128, 127, 300, 2, 0, 513, 64, 1000, 0]
    offsets = torch.tensor([3] + sizes, dtype=torch.int32).cumsum(0).int()
    E, n = len(sizes), int(offsets[-1]) + 2
    rows, cols = (320, 1408)
    q, scale = matrix(rows, cols, 5, groups=E)
    k = rows if back else cols
    x, host = rows_of(n, k, F16, 6)
    xq, xs = to_blocks(host.float())
    y = ctx.block_grouped_linear(x, T.BlockWeight(q.cuda(), scale.cuda()), offsets.cuda(),
                                 transpose=back)
    xd = from_blocks(xq, xs)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            dense = from_blocks(q[e], scale[e], 128)
            check_product(y[a:b], xd[a:b], dense.t() if back else dense, F16, k)
    assert (y[:3] == 0).all() and (y[-2:] == 0).all()


@pytest.mark.parametrize("offsets", [[0, 50, 20, 60], [-5, 10, 40, 500], [60, 60, 0, 0],
                                     [-(1 << 31), 0, (1 << 31) - 1, 5]])
@pytest.mark.parametrize("n", [60, 700])
@pytest.mark.parametrize("back", [False, True])
def test_offsets_that_make_no_sense_stay_inside(T, ctx, offsets, n, back):
    """Unspecified rows of y, and nothing outside it."""
    q, scale = matrix(130, 200, 7, groups=3)
    w = T.BlockWeight(q.cuda(), scale.cuda())
    k, m = (130, 200) if back else (200, 130)
    x, _ = rows_of(n, k, BF, 8)
    out = torch.full((n + 20, m + 5), 3.0, dtype=BF, device="cuda")
    ctx.block_grouped_linear(x, w, torch.tensor(offsets, dtype=torch.int32).cuda(), transpose=back,
                             out=out[10:n + 10, :m])
    torch.cuda.synchronize()
    assert (out[:10] == 3).all() and (out[n + 10:] == 3).all() and (out[:, m:] == 3).all()


def test_more_groups_than_a_launch_holds(T, ctx):
    """Few rows a group of many groups: 65,535 matrices of 520 rows, in two launches."""
    E, rows = 65535, 520
    q = torch.zeros(E, rows, 128, dtype=torch.uint8, device="cuda")
    q[:, :, 0] = 0x38                                      # 1.0
    scale = torch.ones(E, 5, 1, device="cuda")
    w = T.BlockWeight(q.view(E4M3), scale)
    n = 200
    x = torch.zeros(n, 128, dtype=BF, device="cuda")
    x[:, 0] = torch.arange(1, n + 1, device="cuda").to(BF)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[E - 50:] = torch.cat([torch.arange(0, 50), torch.tensor([n])]).int().cuda()
    y = ctx.block_grouped_linear(x, w, offsets)
    assert torch.equal(y, x[:, :1].expand(n, rows))


def test_subnormal_codes_count(T, ctx):
    """Codes below e4m3's normal range, in W and in x."""
    for n in (2, 40, 300):
        q = torch.full((200, 256), 3.0 * 2.0 ** -9).to(E4M3)
        xq = torch.full((n, 256), 2.0 ** -9).to(E4M3)
        one, xs = torch.ones(2, 2), torch.ones(n, 2)
        y = ctx.block_linear(T.BlockRows(xq.cuda(), xs.cuda()), T.BlockWeight(q.cuda(), one.cuda()))
        assert (y.float() == 256 * 3.0 * 2.0 ** -18).all()


def test_a_capture_that_would_grow_the_workspace_is_refused_and_goes_on(T):
    q, s = matrix(260, 384, 111)
    w = T.BlockWeight(q.cuda(), s.cuda())
    x, _ = rows_of(300, 384, BF, 112)
    rows = torch.zeros(4, device="cuda")
    with T.Context(0) as c:
        c.rms_norm(x, torch.ones(384, dtype=BF, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rows += 1
            with pytest.raises(T.Exl3Error) as e:
                c.block_linear(x, w)
        assert e.value.code == T.EXL3_ENOMEM
        graph.replay()
        torch.cuda.synchronize()
        assert (rows == 1).all()
        assert torch.isfinite(c.block_linear(x, w)).all()
        torch.cuda.synchronize()
        del graph


def test_two_products_in_one_graph_and_two_contexts_at_once(T):
    """Calls that share a context's workspace run one after the other; contexts do not meet."""
    q, s = matrix(520, 1024, 121)
    w = T.BlockWeight(q.cuda(), s.cuda())
    xs = [rows_of(n, 1024, BF, 122 + n)[0] for n in (200, 33)]
    with T.Context(0) as a, T.Context(0) as b:
        want = [a.block_linear(x, w) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [[], []]
        for _ in range(4):
            for i, c in enumerate((a, b)):
                with torch.cuda.stream(streams[i]):
                    got[i].append([c.block_linear(x, w) for x in xs])
        torch.cuda.synchronize()
        for side in got:
            for pair in side:
                assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
        # one context on two streams by turns
        for turn in range(4):
            with torch.cuda.stream(streams[turn % 2]):
                y = a.block_linear(xs[0], w)
                z = a.block_linear(xs[1], w)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_a_result_over_the_weight_or_the_offsets_is_refused(T, ctx):
    """And neither is changed; one right behind the codes is written."""
    memory = torch.zeros(256 * 384 + 4 * 256 * 2, dtype=torch.uint8, device="cuda")
    q, s = matrix(256, 384, 131)
    memory[:256 * 384] = q.view(torch.uint8).flatten().cuda()
    scale = torch.zeros(1024, dtype=torch.float32, device="cuda")
    scale[:6] = s.flatten().cuda()
    offsets = torch.zeros(1024, dtype=torch.int32, device="cuda")
    offsets[1] = 4
    w = T.BlockWeight(memory[:256 * 384].view(E4M3).view(256, 384), scale[:6].view(2, 3))
    assert w.q.data_ptr() == memory.data_ptr() and w.scale.data_ptr() == scale.data_ptr()
    x, _ = rows_of(4, 384, BF, 132)
    before = [t.clone() for t in (memory, scale, offsets)]

    def out(t, at):
        return t.view(torch.uint8)[at:at + 2048].view(BF).view(4, 256)
    for over in [out(memory, 0), out(memory, 256 * 384 - 16), out(scale, 0), out(offsets, 0)]:
        for rows in [x, ctx.block_quantize(x)]:
            with pytest.raises(T.Exl3Error) as e:
                ctx.block_grouped_linear(rows, w, offsets[:2], out=over)
            assert e.value.code == T.EXL3_EINVAL
    assert all(torch.equal(a, b) for a, b in zip(before, (memory, scale, offsets)))
    behind = out(memory, 256 * 384)
    ctx.block_linear(x, w, out=behind)
    assert torch.equal(behind, ctx.block_linear(x, w))
    assert torch.equal(memory[:256 * 384], before[0][:256 * 384])
