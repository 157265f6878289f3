"""Products in 8-bit blocks whose two scales multiply to what binary32 does not hold, while the
products of the values themselves do.  Codes are whole numbers times one power of two, so that every
sum is exact and the results are the formula's, rounded once."""
import pytest
import torch

from block_reference import E4M3, blocks, from_blocks, to_blocks

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    with T.Context(0) as c:
        yield c


# (exponents of the rows' scales, of W's scales, what the codes +-1 and 0 are multiplied by)
RANGES = {
    "small": ([-70, -69, -66, -60, -40], -78, 2.0 ** 8),       # their product is subnormal or zero
    "least": ([-126, -120, -110, -100], -22, 2.0 ** 8),        # as those of rows of tiny values
    "large": ([68, 69, 70, -100], 60, 2.0 ** -9),              # infinite
    "high": ([50, 49, 0], 50, 2.0 ** 3),                       # sums above 2^104
    "huge": ([-110, -105, -126], 110, 1.0),                    # one scale large, the other small
    "tiny": ([110, 112, 0], -110, 2.0 ** 3),
    "subnormal": ([-130, -135, -127, -126], 20, 2.0 ** 3),     # scales below the normal range
    "zero": ([None, 0, None, 40], 60, 2.0 ** -9),             # scales of zero
}


def power(e):
    return 0.0 if e is None else 1.25 * 2.0 ** e


def case(which, n, m, k, seed):
    """(x's codes and scales, W's codes and scales): W [m, k], some of its rows empty."""
    rows_e, w_e, unit = RANGES[which]
    g = torch.Generator().manual_seed(seed)
    xq = (torch.randint(-1, 2, (n, k), generator=g).float() * unit).to(E4M3)
    w = torch.randint(-1, 2, (m, k), generator=g).float() * unit
    w[::7] = 0
    at = torch.randint(0, len(rows_e), (n, 1), generator=g).expand(n, blocks(k))
    xs = torch.tensor([power(e) for e in rows_e])[at].contiguous()
    ws = torch.full((blocks(m), blocks(k)), 1.75 * 2.0 ** w_e)
    return xq, xs, w.to(E4M3), ws


def rounded(v):
    return v.float().to(BF)                                # (exact in binary32, so rounded once)


# the streamed form (16-bit rows), and tiles of 32 to 256 columns
SIZES = [(24, 300, 384), (70, 2100, 300), (150, 4096, 1300), (500, 4096, 300), (1500, 4096, 260),
         (3840, 2176, 130)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("which", list(RANGES))
@pytest.mark.parametrize("n,m,k", SIZES)
def test_scales_far_apart(T, ctx, n, m, k, which, back):
    xq, xs, wq, ws = case(which, n, m, k, n + m)
    want = rounded(from_blocks(xq, xs) @ from_blocks(wq, ws, 128).t())
    if back:                                               # W's transpose, contracted over its rows
        wq, ws = wq.t().contiguous(), ws.t().contiguous()
    y = ctx.block_linear(T.BlockRows(xq.cuda(), xs.cuda()), T.BlockWeight(wq.cuda(), ws.cuda()),
                         transpose=back)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("which", list(RANGES))
@pytest.mark.parametrize("k", [384, 2500, 5000])
def test_scales_far_apart_by_group(T, ctx, k, which):
    """Few rows an expert, streamed."""
    E, n, m = 6, 13, 200
    xq, xs, wq, ws = case(which, n, E * 256, k, k)
    wq, ws = wq.view(torch.uint8).view(E, 256, k)[:, :m].contiguous(), ws.view(E, 2, blocks(k))
    offsets = [0, 2, 2, 7, 8, 12, 13]
    y = ctx.block_grouped_linear(T.BlockRows(xq.cuda(), xs.cuda()),
                                 T.BlockWeight(wq.view(E4M3).cuda(), ws.cuda()),
                                 torch.tensor(offsets, dtype=torch.int32).cuda()).cpu()
    x = from_blocks(xq, xs)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        want = rounded(x[a:b] @ from_blocks(wq[e].view(E4M3), ws[e], 128).t())
        assert torch.equal(y[a:b], want)


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("e,w_e", [(-70, -78), (-117, -22), (60, 62)])
def test_rows_in_16_bits(T, ctx, n, e, w_e):
    """Their blocks written in the call: 448 times a power of two has that power as its scale."""
    m, k, unit = 300, 640, 2.0 ** 8 if e < 0 else 2.0 ** -9
    g = torch.Generator().manual_seed(n)
    x = torch.randint(-1, 2, (n, k), generator=g).float() * 7 * 2.0 ** (6 + e)
    x[:, ::128] = 448 * 2.0 ** e
    w = torch.randint(-1, 2, (m, k), generator=g).float() * unit
    w[::7] = 0
    if e > 0:
        w[:, ::128] = 0                                    # (the others' products are in range)
        x[:, 1::2] = 2.0 ** (e - 9)
        x[:, 2::2] = 0
        x[:, ::128] = 448 * 2.0 ** e
    x = x.to(BF)
    xq, xs = to_blocks(x.float())
    assert (xs == 2.0 ** e).all()
    ws = torch.full((blocks(m), blocks(k)), 1.75 * 2.0 ** w_e)
    want = rounded(from_blocks(xq, xs) @ from_blocks(w.to(E4M3), ws, 128).t())
    y = ctx.block_linear(x.cuda(), T.BlockWeight(w.to(E4M3).cuda(), ws.cuda()))
    assert torch.isfinite(want).all() and torch.equal(y.cpu(), want)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n,m,k", SIZES)
def test_rows_of_zeros_leave_the_others_as_they_are(T, ctx, n, m, k, back):
    """Their scale is the smallest, and meets any of W's."""
    g = torch.Generator().manual_seed(k)
    w = ctx.block_quantize_weight((torch.randn((k, m) if back else (m, k), generator=g) * 0.02).cuda())
    x = torch.randn(n, k, generator=g).to(BF).cuda()
    want = ctx.block_linear(ctx.block_quantize(x), w, transpose=back)
    x[1::3] = 0
    want[1::3] = 0
    assert torch.equal(ctx.block_linear(ctx.block_quantize(x), w, transpose=back), want)


def blocks_with_ties():
    """Rows of one block whose largest a is tiny, with values whose quotient by a / 448 lies halfway
    between two codes: 7 * 2^-10 (a * 2^-16) below e4m3's normal range, 21 * 2^j (3 a * 2^i) in it."""
    g = torch.Generator().manual_seed(17)
    rows = []
    for e in list(range(-125, -90)) + [-62, -61, -60, -59, -58, -50, 0, 100]:
        for m in range(128, 256, 3):
            a = m * 2.0 ** (e - 7)
            row = a * (2 * torch.rand(128, generator=g, dtype=torch.float64) - 1)
            row[0] = a
            for i in range(8):
                row[1 + i] = (-1) ** i * a * 2.0 ** -(16 - i)
                row[20 + i] = (-1) ** i * 3 * a * 2.0 ** -(6 + i)
            rows.append(row)
    return torch.stack(rows).float()


def same(got, want):
    return torch.equal(got.cpu().contiguous().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_codes_of_tiny_blocks_are_those_of_a_division(ctx, dtype):
    v = blocks_with_ties().to(dtype)
    if dtype == BF:
        q, scale = to_blocks(v.float())
        got = ctx.block_quantize(v.cuda())
        assert torch.equal(got.scale.cpu(), scale) and same(got.q, q)
        # and where the product's workgroups write the rows themselves: times a multiple of the unit
        # matrix, each result one code times two scales
        one = torch.eye(128).to(E4M3).cuda()
        w = ctx_weight(one, 2.0 ** 60)
        for t in range(0, v.shape[0], 97):
            y = ctx.block_linear(v[t:t + 1].cuda(), w)
            want = (from_blocks(q[t:t + 1], scale[t:t + 1]) * 2.0 ** 60).float().to(BF)
            assert torch.equal(y.cpu(), want)
    # matrices: a row's values one to a row of its own, 128 x 128 with the same largest
    for t in range(0, v.shape[0], 53):
        w = v[t:t + 1].expand(128, 128).contiguous()
        q, scale = to_blocks(w.float(), 128)
        got = ctx.block_quantize_weight(w.cuda())
        assert torch.equal(got.scale.cpu(), scale) and same(got.q, q)


def ctx_weight(codes, scale):
    from trellis_coded_weight_amd import BlockWeight
    return BlockWeight(codes, torch.full((1, 1), scale, device="cuda"))


@pytest.mark.parametrize("cols", [1, 130, 300, 1003, 20001])
def test_codes_behind_a_row_are_zero_also_after_a_nan(ctx, cols):
    """Up to whole blocks, as products read them."""
    x = torch.ones(3, cols, dtype=BF)
    x[1, cols - 1] = float("nan")
    x = x.cuda()
    gain = torch.ones(cols, dtype=BF, device="cuda")
    for got in (ctx.block_quantize(x), ctx.rms_norm(x, gain, blocks=True),
                ctx.block_quantize_weight(x)):
        codes = got.q.as_strided((3, 128 * blocks(cols)), (128 * blocks(cols), 1))
        codes = codes.view(torch.uint8)
        assert (codes[:, cols:] == 0).all()
        assert (codes[1, cols - 1] & 0x7F) == 0x7F
        assert torch.isnan(got.scale[-1 if got.scale.shape[0] == 1 else 1, -1])


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("which", list(RANGES))
@pytest.mark.parametrize("n,m,k", [(60, 130, 300), (1500, 260, 300), (4000, 520, 600)])
def test_scales_far_apart_by_group_in_tiles(T, ctx, n, m, k, which, back):
    E = 3
    xq, xs, wq, ws = case(which, n, E * 640, k, n + k)
    wq = wq.view(torch.uint8).view(E, 640, k)[:, :m].contiguous()
    ws = ws.view(E, 5, blocks(k))[:, :blocks(m)].contiguous()
    if back:
        wq, ws = wq.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous()
    offsets = [1, n // 3, n // 3, n - 2]
    y = ctx.block_grouped_linear(T.BlockRows(xq.cuda(), xs.cuda()),
                                 T.BlockWeight(wq.view(E4M3).cuda(), ws.cuda()),
                                 torch.tensor(offsets, dtype=torch.int32).cuda(),
                                 transpose=back).cpu()
    x = from_blocks(xq, xs)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        w = from_blocks(wq[e].view(E4M3), ws[e], 128)
        assert torch.equal(y[a:b], rounded(x[a:b] @ (w if back else w.t())))
    assert (y[:1] == 0).all() and (y[n - 2:] == 0).all()
