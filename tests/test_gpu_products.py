"""Products with coded weights (linear, grouped by expert, low-rank adapters) on the GPU against
64-bit products of the oracle's dequantized matrices."""
import ctypes

import numpy as np
import pytest
import torch

from product_reference import HALF, check, dense, inner_of, random_weight, spread_of

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    c = T.Context(0)
    yield c
    c.close()


@pytest.fixture(scope="module")
def ctx_of(T):
    made = {}

    def get(codebook):
        if codebook not in made:
            made[codebook] = T.Context(0)
            made[codebook].set_codebook_kind(codebook)
        return made[codebook]

    yield get
    for c in made.values():
        c.close()


def on_gpu(T, w):
    scale = torch.from_numpy(np.atleast_1d(w["scale"])).to(DEV)
    return T.CodedWeight(torch.from_numpy(w["packed"]).to(DEV), w["K"], scale,
                         torch.from_numpy(w["su"]).to(DEV), torch.from_numpy(w["sv"]).to(DEV),
                         had_block=w["had"])


def rows_of(n, k, dtype, seed, std=1.0):
    """Activations with a few large channels, exact in `dtype`: (tensor, float64 array)."""
    r = np.random.Generator(np.random.PCG64(seed))
    x = r.standard_normal((n, k)) * np.where(r.random(k) < 0.02, 10.0, 1.0) * std
    t = torch.from_numpy(x).to(dtype)
    return t.to(DEV), t.double().numpy()


# ---- levels ----
# A stream whose 16 K = 64 bits a row repeat one 16-bit word gives every row of a tile the same
# states, the word's rotations by 4 bits.  An input that is a row of H picks one column, whose
# 128 times the level in every row, transformed (with factors 128^-1/2 twice): the output is 128 levels
# in the block's first row, exactly.  The words are one of each class of rotations, so every state is met.
@pytest.mark.parametrize("codebook", ["mul1", "mcg", "3inst"])
def test_levels_of_all_states(T, ctx_of, codebook):
    import scipy.linalg

    import oracle
    words = np.arange(65536)
    rot = np.stack([((words << (4 * i)) | (words >> (16 - 4 * i))) & 0xFFFF for i in range(4)])
    words = words[words == rot.min(axis=0)]
    groups = -(-len(words) // 16)
    words = np.resize(words, groups * 16).reshape(groups, 16)
    packed = np.repeat(np.repeat(words[:, None, :, None], 8, 1), 64, 3).astype(np.uint16)
    h = scipy.linalg.hadamard(128).astype(np.float32)
    x = np.zeros((64, 256), np.float32)
    cols = [16 * (i // 4) + i % 4 for i in range(64)]
    for i, c in enumerate(cols):
        x[i, c // 128 * 128:c // 128 * 128 + 128] = h[c % 128]
    w = T.CodedWeight(torch.from_numpy(packed.view(np.int16)).to(DEV), 4,
                      torch.ones(groups, device=DEV), torch.ones(groups, 128, device=DEV),
                      torch.ones(groups, 256, device=DEV))
    xs = torch.from_numpy(x).half().to(DEV).repeat(groups, 1)
    offsets = torch.arange(groups + 1, dtype=torch.int32, device=DEV) * 64
    y = ctx_of(codebook).grouped_linear(xs, w, offsets).float().cpu().numpy()
    lv = {"mul1": oracle.mul1_levels_fp16, "mcg": oracle.mcg_levels_fp16,
          "3inst": oracle.inst3_levels_fp16}[codebook]()
    lv = np.asarray(lv).view(np.float16).astype(np.float32)
    states = oracle.unpack_states(packed[:, 0].reshape(-1, 64), 4)[:, :4].reshape(groups, 64)
    assert len(np.unique(states)) == 65536
    assert np.array_equal(y[:, 0].reshape(groups, 64), 128 * lv[states])
    assert (y[:, 1:] == 0).all()


# ---- linear ----
SHAPES = [
    # n, rows, cols, K, had, dtype, codebook
    (1, 128, 128, 2, 128, BF, "mul1"),
    (1, 256, 1152, 1, 128, FP, "mul1"),
    (2, 192, 320, 3, 64, FP, "mul1"),
    (15, 384, 2176, 4, 128, BF, "mcg"),
    (16, 128, 512, 2, 64, BF, "3inst"),
    (17, 640, 256, 3, 128, BF, "3inst"),
    (33, 64, 64, 1, 64, FP, "mcg"),
    (63, 256, 384, 4, 64, FP, "mul1"),
    (64, 1280, 128, 2, 128, FP, "3inst"),
    (65, 128, 1152, 3, 128, BF, "mul1"),
    (129, 192, 192, 4, 64, FP, "3inst"),
    (257, 384, 256, 1, 128, BF, "mul1"),
    (300, 640, 576, 2, 64, BF, "mcg"),
    (1030, 1152, 384, 2, 128, FP, "mul1"),
    (5, 256, 256, 5, 128, BF, "mul1"),
    (200, 128, 256, 8, 128, FP, "mul1"),
]


@pytest.mark.parametrize("n,rows,cols,K,had,dtype,codebook", SHAPES)
@pytest.mark.parametrize("transpose", [False, True])
def test_linear(T, ctx_of, n, rows, cols, K, had, dtype, codebook, transpose):
    w = random_weight(rows, cols, K, had, n + rows + K)
    m = dense(w, codebook)
    m = m.T if transpose else m
    x, x64 = rows_of(n, m.shape[1], dtype, n + cols)
    y = ctx_of(codebook).linear(x, on_gpu(T, w), transpose=transpose)
    assert y.shape == (n, m.shape[0]) and y.dtype == dtype
    # the looser of the two forms' bounds: which one runs is a matter of speed
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(False, dtype))


def test_large_tile(T, ctx):
    """Sizes that fill the chip with the largest tile, with edges on both sides."""
    w = random_weight(4096 + 128, 384, 2, 128, 71)
    x, x64 = rows_of(2100, 384, BF, 72)
    m = dense(w)
    check(ctx.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(False, BF))


def test_both_forms_agree(T, ctx):
    """The same rows, few at a time and all at once."""
    w = random_weight(256, 640, 3, 128, 81)
    x, x64 = rows_of(96, 640, FP, 82)
    g, m = on_gpu(T, w), dense(w)
    parts = torch.cat([ctx.linear(x[i:i + 7], g) for i in range(0, 96, 7)])
    want, spread = x64 @ m.T, spread_of(x64, m)
    check(parts, want, spread, inner_of(True, FP))
    check(ctx.linear(x, g), want, spread, inner_of(False, FP))


@pytest.mark.parametrize("n", [3, 150])
def test_tile_order_and_own_table(T, n):
    r = np.random.Generator(np.random.PCG64(91))
    order = r.permutation(256).astype(np.uint8)
    table = (r.standard_normal(65536)).astype(np.float16)
    w = random_weight(128, 256, 2, 64, 92)
    x, x64 = rows_of(n, 256, BF, 93)
    with T.Context(0) as c:
        c.set_tile_order(order)
        m = dense(w, "mul1", order)
        check(c.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(False, BF))
        c.set_codebook(torch.from_numpy(table))
        m = dense(w, table, order)
        check(c.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(False, BF))
        c.set_tile_order(None)
        m = dense(w, table)
        check(c.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(False, BF))
        c.set_codebook(None)
        m = dense(w, "mul1")
        check(c.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(False, BF))


def test_quantized_matrix_end_to_end(T, ctx):
    """quantize_matrix's container through linear is the product with the dequantized matrix."""
    import workloads
    mt = workloads.gaussian(256, 384, 0.02, 5, 6, K=2)
    su, sv = torch.from_numpy(mt.su).to(DEV), torch.from_numpy(mt.sv).to(DEV)
    out = ctx.quantize_matrix(torch.from_numpy(mt.w).to(DEV).bfloat16(), 2, su, sv)
    tiles = ctx.decode_tiles(out["packed"].reshape(-1, 32), 2, out["scale"])
    m = ctx.unregularize(tiles, 256, 384, su, sv).double().cpu().numpy()
    x, x64 = rows_of(9, 384, BF, 7)
    g = T.CodedWeight(out["packed"], 2, out["scale"], su, sv)
    check(ctx.linear(x, g), x64 @ m.T, spread_of(x64, m), inner_of(True, BF))


@pytest.mark.parametrize("n", [1, 6, 90])
@pytest.mark.parametrize("shift,pitch", [(0, 640), (1, 643), (8, 648), (3, 1000)])
def test_pitch_and_alignment(T, ctx, n, shift, pitch):
    w = random_weight(256, 384, 2, 128, 101)
    m = dense(w)
    x, x64 = rows_of(n, 384, FP, 102)
    big = torch.full((n, pitch), 777.0, dtype=FP, device=DEV)
    flat = torch.full((n * pitch + 16,), 555.0, dtype=FP, device=DEV)
    xin = torch.as_strided(big, (n, 384), (pitch, 1), shift) if shift + 384 <= pitch else None
    xin.copy_(x)
    out = torch.as_strided(flat, (n, 256), (pitch, 1), shift)
    assert ctx.linear(xin, on_gpu(T, w), out=out) is out
    check(out, x64 @ m.T, spread_of(x64, m), inner_of(False, FP))
    left = flat.cpu().numpy().astype(np.float32)
    for t in range(n):
        left[t * pitch + shift:t * pitch + shift + 256] = 555.0
    assert (left == 555.0).all(), "written outside the rows"


def test_interleaved_input_and_output(T, ctx):
    w = random_weight(128, 256, 2, 128, 111)
    m = dense(w)
    x, x64 = rows_of(80, 256, BF, 112)
    both = torch.zeros(80, 384, dtype=BF, device=DEV)
    both[:, :256] = x
    ctx.linear(both[:, :256], on_gpu(T, w), out=both[:, 256:])
    check(both[:, 256:], x64 @ m.T, spread_of(x64, m), inner_of(False, BF))
    assert torch.equal(both[:, :256], x)


def test_rows_that_are_not_contiguous_are_copied(T, ctx):
    w = random_weight(128, 256, 2, 128, 121)
    m = dense(w)
    x, x64 = rows_of(4, 256, BF, 122)
    y = ctx.linear(x.t().contiguous().t(), on_gpu(T, w))
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(True, BF))


@pytest.mark.parametrize("std", [1e30, 1e-30])
def test_range_of_bfloat16(T, ctx, std):
    w = random_weight(128, 512, 2, 128, 131)
    m = dense(w)
    x, x64 = rows_of(3, 512, BF, 132, std)
    y = ctx.linear(x, on_gpu(T, w)).double() / std
    check(y, x64 / std @ m.T, spread_of(x64 / std, m), inner_of(True, BF))


@pytest.mark.parametrize("n", [8, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_row_stays_alone(T, ctx, n, bad):
    w = random_weight(256, 384, 2, 128, 141)
    x, _ = rows_of(n, 384, BF, 142)
    g = on_gpu(T, w)
    clean = ctx.linear(x, g)
    x[5, 200] = bad
    y = ctx.linear(x, g)
    assert not torch.isfinite(y[5]).any()
    keep = torch.arange(n, device=DEV) != 5
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("n", [8, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_alone_in_the_other_direction(T, ctx, n, bad):
    w = random_weight(384, 256, 3, 128, 145)
    x, _ = rows_of(n, 384, BF, 146)
    g = on_gpu(T, w)
    clean = ctx.linear(x, g, transpose=True)
    x[5, 200] = bad
    y = ctx.linear(x, g, transpose=True)
    assert not torch.isfinite(y[5]).any()
    keep = torch.arange(n, device=DEV) != 5
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("n,per", [(1, 0), (31, 0), (3, 4), (90, 40)])
@pytest.mark.parametrize("K,codebook", [(1, "mul1"), (2, "mcg"), (3, "mul1"), (4, "3inst")])
def test_the_other_direction_in_tiles_meets_the_dense_form(T, ctx_of, n, per, K, codebook):
    """Words that start on 8 bytes take the dense weights, aligned ones the tiles: both are within
    their bounds of the 64-bit product.  Rows long enough to be split; the last tile of columns
    is partly filled."""
    groups = 3 if per else None
    w = random_weight(2176, 192, K, 64, 147 + K, groups=groups)
    c, g = ctx_of(codebook), on_gpu(T, w)
    flat = torch.zeros(g.packed.numel() + 4, dtype=torch.int16, device=DEV)
    flat[4:] = g.packed.reshape(-1)
    h = T.CodedWeight(flat[4:].view(g.packed.shape), K, g.scale, g.su, g.sv, had_block=64)
    assert h.packed.data_ptr() % 16 == 8
    x, x64 = rows_of(n, 2176, FP, 148)
    if groups is None:
        m = dense(w, codebook).T
        for u in (g, h):
            check(c.linear(x, u, transpose=True), x64 @ m.T, spread_of(x64, m), inner_of(False, FP))
        return
    cut = np.array([0, n - per if n > per else 1, n - 1, n], np.int32)
    at = torch.from_numpy(cut).to(DEV)
    for u in (g, h):
        y = c.grouped_linear(x, u, at, transpose=True)
        for e in range(3):
            m, xe = dense(w, codebook, group=e).T, x64[cut[e]:cut[e + 1]]
            check(y[cut[e]:cut[e + 1]], xe @ m.T, spread_of(xe, m), inner_of(False, FP), "%d" % e)


@pytest.mark.parametrize("n", [600, 1536, 1537])
@pytest.mark.parametrize("transpose", [False, True])
def test_long_contractions_of_many_rows(T, ctx, n, transpose):
    w = random_weight(2624, 192, 2, 64, n) if transpose else random_weight(192, 2624, 2, 64, n)
    m = dense(w).T if transpose else dense(w)
    x, x64 = rows_of(n, 2624, BF, n + 1)
    y = ctx.linear(x, on_gpu(T, w), transpose=transpose)
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(False, BF))


def test_zero_rows_and_zero_input(T, ctx):
    w = random_weight(128, 256, 2, 128, 151)
    g = on_gpu(T, w)
    assert ctx.linear(torch.empty(0, 256, dtype=BF, device=DEV), g).shape == (0, 128)
    for n in (2, 100):
        y = ctx.linear(torch.zeros(n, 256, dtype=BF, device=DEV), g)
        assert (y == 0).all()


# ---- grouped ----
GROUPED = [
    # sizes, rows, cols, K, had, dtype
    ([3, 0, 5, 1, 0, 0, 2], 128, 256, 2, 128, BF),
    ([0, 0, 9], 192, 128, 3, 64, FP),
    ([1] * 70, 64, 128, 2, 64, BF),
    ([40, 0, 0, 2], 256, 384, 4, 128, FP),
    ([130, 0, 301, 7, 64], 256, 384, 2, 128, BF),
    ([0, 500, 0, 0], 128, 128, 1, 64, FP),
    ([17] * 20 + [400] + [0] * 50, 128, 256, 3, 128, BF),
]


@pytest.mark.parametrize("sizes,rows,cols,K,had,dtype", GROUPED)
@pytest.mark.parametrize("transpose", [False, True])
def test_grouped(T, ctx, sizes, rows, cols, K, had, dtype, transpose):
    w = random_weight(rows, cols, K, had, sum(sizes), groups=len(sizes))
    n = sum(sizes)
    x, x64 = rows_of(n, rows if transpose else cols, dtype, n + 1)
    cut = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = ctx.grouped_linear(x, on_gpu(T, w), torch.from_numpy(cut).to(DEV), transpose=transpose)
    for e in range(len(sizes)):
        if sizes[e]:
            m = dense(w, group=e)
            m = m.T if transpose else m
            xe = x64[cut[e]:cut[e + 1]]
            check(y[cut[e]:cut[e + 1]], xe @ m.T, spread_of(xe, m), inner_of(False, dtype),
                  "group %d" % e)


@pytest.mark.parametrize("per", [2, 150])
@pytest.mark.parametrize("transpose", [False, True])
def test_rows_of_no_group_are_zero(T, ctx, per, transpose):
    w = random_weight(128, 128, 2, 64, 161, groups=3)
    n = 3 * per + 9
    x, x64 = rows_of(n, 128, BF, 162)
    cut = np.array([4, 4 + per, 4 + per, 4 + 3 * per], np.int32)
    y = ctx.grouped_linear(x, on_gpu(T, w), torch.from_numpy(cut).to(DEV), transpose=transpose)
    assert (y[:4] == 0).all() and (y[cut[3]:] == 0).all()
    for e in (0, 2):
        m = dense(w, group=e)
        m = m.T if transpose else m
        xe = x64[cut[e]:cut[e + 1]]
        check(y[cut[e]:cut[e + 1]], xe @ m.T, spread_of(xe, m), inner_of(False, BF))


def test_groups_in_batches_of_the_scratch_bound(T, ctx):
    """A scratch bound of two dense matrices takes the groups two at a time, with equal results."""
    w = random_weight(128, 256, 2, 128, 171, groups=7)
    x, _ = rows_of(900, 256, BF, 172)
    cut = torch.tensor([0, 200, 201, 400, 400, 650, 800, 900], dtype=torch.int32, device=DEV)
    want = ctx.grouped_linear(x, on_gpu(T, w), cut)
    with T.Context(0, scratch_bytes=2 * 128 * 256 * 2) as small:
        got = small.grouped_linear(x, on_gpu(T, w), cut)
        torch.cuda.synchronize()
    assert torch.equal(got, want)


# ---- adapters ----
def adapters_of(T, rows, cols, count, rank, dtype, seed):
    r = np.random.Generator(np.random.PCG64(seed))
    A = torch.from_numpy(r.standard_normal((count, rank, cols)) / np.sqrt(cols)).to(dtype)
    B = torch.from_numpy(r.standard_normal((count, rows, rank)) * 0.1).to(dtype)
    al = torch.from_numpy((0.5 + r.random(count)).astype(np.float32))
    return (T.Adapters(A.to(DEV), B.to(DEV), al.to(DEV)), A.double().numpy(), B.double().numpy(),
            al.double().numpy())


def adapter_forward(x, A, B, al, ids):
    """The adapters' part, and the root of the sum of squares of its last contraction's terms."""
    y, s = np.zeros((len(x), B.shape[1])), np.zeros((len(x), B.shape[1]))
    for t, a in enumerate(ids):
        if 0 <= a < len(al):
            v = al[a] * (A[a] @ x[t])
            y[t], s[t] = B[a] @ v, np.sqrt((B[a] ** 2) @ (v ** 2))
    return y, s


ADAPTERS = [
    # n, rows, cols, K, had, dtype, count, rank
    (1, 128, 256, 2, 128, BF, 3, 8),
    (7, 256, 128, 3, 64, FP, 5, 1),
    (32, 256, 384, 2, 128, BF, 32, 16),
    (50, 128, 128, 4, 128, FP, 2, 5),
    (64, 192, 256, 2, 64, BF, 40, 33),
    (70, 256, 256, 1, 128, FP, 4, 12),
    (150, 384, 128, 2, 128, BF, 3, 128),
    (333, 256, 640, 2, 128, FP, 9, 64),
    (600, 4096, 128, 2, 128, BF, 5, 100),
]


def ids_of(n, count, seed):
    """Runs of rows of one adapter, some without, and one value out of range."""
    r = np.random.Generator(np.random.PCG64(seed))
    ids = np.repeat(r.integers(-1, count, n), r.integers(1, max(2, n // 8), n))[:n].astype(np.int32)
    if n > 4:
        ids[n // 2] = count + 3
        ids[n // 3] = -7
    return ids


@pytest.mark.parametrize("n,rows,cols,K,had,dtype,count,rank", ADAPTERS)
def test_adapter_linear(T, ctx, n, rows, cols, K, had, dtype, count, rank):
    w = random_weight(rows, cols, K, had, n)
    ad, A, B, al = adapters_of(T, rows, cols, count, rank, dtype, n + 1)
    x, x64 = rows_of(n, cols, dtype, n + 2)
    ids = ids_of(n, count, n + 3)
    y = ctx.adapter_linear(x, on_gpu(T, w), ad, torch.from_numpy(ids).to(DEV))
    m = dense(w)
    part, s = adapter_forward(x64, A, B, al, ids)
    # v's rounding is one more half step of the adapters' terms
    check(y, x64 @ m.T + part, spread_of(x64, m) + s, inner_of(False, dtype))


# sizes at which each tile of the matrix product takes the fewest rounds of 256 compute units, none
# of them a multiple of the tile
TILES = [(1450, 1470, 4032), (700, 2900, 4032), (901, 1500, 4160), (5, 4000, 4032)]


@pytest.mark.parametrize("seed,n,rows", TILES)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_every_tile_of_the_matrix_product(T, ctx, seed, n, rows, dtype):
    """With the shortest contractions, alone and with adapters of an unaligned rank."""
    cols = 64 if dtype is BF else 192
    w = random_weight(rows, cols, 2, 64, seed)
    g, m = on_gpu(T, w), dense(w)
    x, x64 = rows_of(n, cols, dtype, seed + 1)
    check(ctx.linear(x, g), x64 @ m.T, spread_of(x64, m), inner_of(False, dtype))
    ad, A, B, al = adapters_of(T, rows, cols, 3, 7, dtype, seed + 2)
    ids = ids_of(n, 3, seed + 3)
    y = ctx.adapter_linear(x, g, ad, torch.from_numpy(ids).to(DEV))
    part, s = adapter_forward(x64, A, B, al, ids)
    check(y, x64 @ m.T + part, spread_of(x64, m) + s, inner_of(False, dtype))


@pytest.mark.parametrize("n", [20, 200])
def test_a_bad_adapter_stays_alone(T, ctx, n):
    """NaN and infinity in one adapter reach its own rows only."""
    w = random_weight(128, 256, 2, 128, 181)
    ad, *_ = adapters_of(T, 128, 256, 3, 8, BF, 182)
    x, _ = rows_of(n, 256, BF, 183)
    ids = torch.arange(n, dtype=torch.int32, device=DEV) % 4 - 1
    clean = ctx.adapter_linear(x, on_gpu(T, w), ad, ids)
    ad.A[1, 2, 7] = float("nan")
    ad.B[1, :, 3] = float("inf")
    y = ctx.adapter_linear(x, on_gpu(T, w), ad, ids)
    assert torch.equal(y[ids != 1], clean[ids != 1])
    assert not torch.isfinite(y[ids == 1]).any()
    dy, _ = rows_of(n, 128, BF, 184)
    dx, dA, dB = ctx.adapter_linear_backward(dy, x, on_gpu(T, w), ad, ids)
    assert torch.isfinite(dx[ids != 1]).all()
    for a in (0, 2):
        assert torch.isfinite(dA[a]).all() and torch.isfinite(dB[a]).all()


def test_a_bad_row_stays_out_of_other_adapters_gradients(T, ctx):
    w = random_weight(128, 128, 2, 64, 191)
    ad, *_ = adapters_of(T, 128, 128, 2, 4, FP, 192)
    x, _ = rows_of(90, 128, FP, 193)
    dy, _ = rows_of(90, 128, FP, 194, 0.01)
    ids = torch.arange(90, dtype=torch.int32, device=DEV) % 2
    clean = ctx.adapter_linear_backward(dy, x, on_gpu(T, w), ad, ids)
    x[4] = float("nan")
    dy[6] = float("inf")
    got = ctx.adapter_linear_backward(dy, x, on_gpu(T, w), ad, ids)
    for c, g in zip(clean[1:], got[1:]):
        assert torch.equal(c[1], g[1])
    keep = torch.arange(90, device=DEV) != 6
    assert torch.equal(clean[0][keep], got[0][keep])


@pytest.mark.parametrize("n,rows,cols,K,had,dtype,count,rank", ADAPTERS)
def test_adapter_backward(T, ctx, n, rows, cols, K, had, dtype, count, rank):
    w = random_weight(rows, cols, K, had, n)
    ad, A, B, al = adapters_of(T, rows, cols, count, rank, dtype, n + 1)
    x, x64 = rows_of(n, cols, dtype, n + 2)
    dy, d64 = rows_of(n, rows, dtype, n + 4, 0.05)
    ids = ids_of(n, count, n + 3)
    dx, dA, dB = ctx.adapter_linear_backward(dy, x, on_gpu(T, w), ad,
                                             torch.from_numpy(ids).to(DEV))
    m = dense(w)
    part, s = adapter_forward(d64, B.transpose(0, 2, 1), A.transpose(0, 2, 1), al, ids)
    check(dx, d64 @ m + part, spread_of(d64, m.T) + s, inner_of(False, dtype), "dx")
    for a in range(count):
        at = np.flatnonzero(ids == a)
        v, u = al[a] * (x64[at] @ A[a].T), al[a] * (d64[at] @ B[a])
        half = (HALF[dtype], dtype)
        check(dA[a], u.T @ x64[at], np.sqrt((u ** 2).T @ x64[at] ** 2), half, "dA")
        check(dB[a], d64[at].T @ v, np.sqrt((d64[at] ** 2).T @ v ** 2), half, "dB")


def test_gradients_against_differences(T, ctx):
    """The forward pass is linear in each of x, A and B: a change of one changes sum(dy y) by
    the gradient's product with it, here with the forward pass in 64 bits."""
    n, rows, cols, count, rank = 75, 128, 192, 3, 6
    w = random_weight(rows, cols, 2, 64, 201)
    ad, A, B, al = adapters_of(T, rows, cols, count, rank, FP, 202)
    x, x64 = rows_of(n, cols, FP, 203)
    dy, d64 = rows_of(n, rows, FP, 204)
    ids = ids_of(n, count, 205)
    got = ctx.adapter_linear_backward(dy, x, on_gpu(T, w), ad, torch.from_numpy(ids).to(DEV))
    m = dense(w)

    def loss(x, A, B):
        return float((d64 * (x @ m.T + adapter_forward(x, A, B, al, ids)[0])).sum())

    r = np.random.Generator(np.random.PCG64(206))
    base = loss(x64, A, B)
    for i, p in enumerate((x64, A, B)):
        step = r.standard_normal(p.shape)
        args = [x64, A, B]
        args[i] = p + step
        diff = loss(*args) - base
        g = got[i].double().cpu().numpy()
        # the gradient's values are off by at most a few half steps of themselves and of the
        # terms inside; the product with an independent step averages them
        tol = 8 * 3 * HALF[FP] * np.linalg.norm(g)
        assert abs((g * step).sum() - diff) <= tol


def test_parts_of_the_backward_pass(T, ctx):
    w = random_weight(128, 256, 2, 128, 211)
    ad, *_ = adapters_of(T, 128, 256, 2, 8, BF, 212)
    x, _ = rows_of(100, 256, BF, 213)
    dy, _ = rows_of(100, 128, BF, 214)
    ids = torch.from_numpy(ids_of(100, 2, 215)).to(DEV)
    g = on_gpu(T, w)
    dx, dA, dB = ctx.adapter_linear_backward(dy, x, g, ad, ids)
    only = ctx.adapter_linear_backward(dy, x, g, ad, ids, want_adapters=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    rest = ctx.adapter_linear_backward(dy, x, g, ad, ids, want_dx=False)
    assert rest[0] is None and torch.equal(rest[1], dA) and torch.equal(rest[2], dB)
    none = ctx.adapter_linear_backward(dy[:0], x[:0], g, ad, ids[:0])
    assert none[0].shape == (0, 256) and (none[1] == 0).all() and (none[2] == 0).all()


# ---- streams, graphs, repeats ----
def _calls(T, n):
    w = on_gpu(T, random_weight(256, 384, 2, 128, 221))
    we = on_gpu(T, random_weight(256, 384, 2, 128, 222, groups=3))
    ad, *_ = adapters_of(T, 256, 384, 4, 8, BF, 223)
    cut = torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device=DEV)
    ids = torch.from_numpy(ids_of(n, 4, 224)).to(DEV)

    def run(c, x, dy):
        return [c.linear(x, w), c.linear(dy, w, transpose=True), c.grouped_linear(x, we, cut),
                c.grouped_linear(dy, we, cut, transpose=True), c.adapter_linear(x, w, ad, ids),
                *c.adapter_linear_backward(dy, x, w, ad, ids)]
    return run


@pytest.mark.parametrize("n", [3, 12, 300])
def test_repeats_are_bit_equal_on_any_stream(T, n):
    run = _calls(T, n)
    x, _ = rows_of(n, 384, BF, 225)
    dy, _ = rows_of(n, 256, BF, 226)
    with T.Context(0) as c:
        first = run(c, x, dy)
        second = run(c, x, dy)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            third = run(c, x, dy)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("n", [3, 12, 300])
def test_graph_replays(T, n):
    run = _calls(T, n)
    c = T.Context(0)
    side = torch.cuda.Stream()
    x, _ = rows_of(n, 384, BF, 235)
    dy, _ = rows_of(n, 256, BF, 236)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(c, x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run(c, x, dy)
    with T.Context(0) as other:
        for seed in range(4):
            xn, _ = rows_of(n, 384, BF, 240 + seed)
            dn, _ = rows_of(n, 256, BF, 250 + seed)
            want = run(other, xn, dn)
            x.copy_(xn)
            dy.copy_(dn)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)
    # a larger call outgrows the workspace; the graph's own stays
    wide, _ = rows_of(4 * n, 384, BF, 260)
    w = on_gpu(T, random_weight(1024, 384, 2, 128, 261))
    with torch.cuda.stream(side):
        c.linear(wide, w)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    del graph
    c.close()


def test_growth_during_a_capture_is_refused(T):
    w = on_gpu(T, random_weight(128, 128, 2, 128, 271))
    x, _ = rows_of(4, 128, BF, 272)
    c = T.Context(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        small, _ = rows_of(1, 128, BF, 273)
        c.linear(small, w)
    big, _ = rows_of(4000, 128, BF, 274)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = c.linear(small, w)
        with pytest.raises(T.Exl3Error) as e:
            c.linear(big, w)
    assert e.value.code == T.EXL3_ENOMEM and "capture" in e.value.msg
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()
    del graph
    c.close()


# ---- refusals ----
def test_refusals_leave_the_output(T, ctx):
    w = on_gpu(T, random_weight(128, 256, 2, 128, 281))
    x = torch.zeros(4, 256, dtype=BF, device=DEV)
    y = torch.full((4, 128), 3.0, dtype=BF, device=DEV)
    lib, vp = ctx.lib, ctypes.c_void_p
    ctx._sync_stream()

    def call(weight=w._ref, xp=x.data_ptr(), ldx=256, n=4, dtype=T.EXL3_BF16, yp=y.data_ptr(),
             ldy=128, transpose=0):
        return lib.exl3_linear(ctx.handle, weight, transpose, xp, ldx, n, dtype, yp, ldy)

    def changed(**kw):
        c = type(w._c).from_buffer_copy(w._c)
        for k, v in kw.items():
            setattr(c, k, v)
        return ctypes.byref(c)

    E, U = T.EXL3_EINVAL, T.EXL3_EUNSUPPORTED
    host = torch.zeros(4, 256, dtype=BF)
    for want, kw in [
            (E, {"weight": None}), (E, {"xp": None}), (E, {"yp": None}), (E, {"ldx": 255}),
            (E, {"ldy": 127}), (E, {"n": -1}), (E, {"n": 1 << 25}), (E, {"dtype": T.EXL3_F32}),
            (E, {"xp": host.data_ptr()}), (E, {"xp": x.data_ptr() + 1}),
            (E, {"yp": x.data_ptr()}), (E, {"n": 1 << 24}),
            (E, {"weight": changed(packed=None)}), (E, {"weight": changed(scale=None)}),
            (E, {"weight": changed(rows=100)}), (E, {"weight": changed(cols=0)}),
            (E, {"weight": changed(groups=0)}), (E, {"weight": changed(groups=2)}),
            (E, {"weight": changed(packed=w.packed.data_ptr() + 2)}),
            (E, {"weight": changed(rows=1 << 20)}),
            (U, {"weight": changed(K=9)}), (U, {"weight": changed(K=0)}),
            (U, {"weight": changed(had_block=32)})]:
        assert call(**kw) == want, kw
        assert ctx.last_error()
    assert lib.exl3_linear(None, w._ref, 0, x.data_ptr(), 256, 4, T.EXL3_BF16, y.data_ptr(),
                           128) == E
    assert lib.exl3_grouped_linear(ctx.handle, w._ref, None, 0, x.data_ptr(), 256, 4,
                                   T.EXL3_BF16, y.data_ptr(), 128) == E
    short = torch.zeros(1, dtype=torch.int32)
    assert lib.exl3_grouped_linear(ctx.handle, w._ref, short.data_ptr(), 0, x.data_ptr(), 256, 4,
                                   T.EXL3_BF16, y.data_ptr(), 128) == E
    ad, *_ = adapters_of(T, 128, 256, 2, 8, BF, 282)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)

    def adapter(adp=ad._ref, idp=ids.data_ptr(), weight=w._ref):
        return lib.exl3_adapter_linear(ctx.handle, weight, adp, idp, x.data_ptr(), 256, 4,
                                       T.EXL3_BF16, y.data_ptr(), 128)

    def other(**kw):
        c = type(ad._c).from_buffer_copy(ad._c)
        for k, v in kw.items():
            setattr(c, k, v)
        return ctypes.byref(c)

    for want, kw in [(E, {"adp": None}), (E, {"idp": None}), (E, {"adp": other(a=None)}),
                     (E, {"adp": other(count=0)}), (U, {"adp": other(rank=0)}),
                     (U, {"adp": other(rank=129)}), (E, {"adp": other(count=60000)}),
                     (E, {"weight": changed(groups=2)})]:
        assert adapter(**kw) == want, kw
    torch.cuda.synchronize()
    assert (y == 3.0).all()
    with T.Context(0, scratch_bytes=1000) as tiny:
        wide = torch.zeros(1000, 128, dtype=BF, device=DEV)      # rows that take dense weights
        with pytest.raises(T.Exl3Error) as e:
            tiny.linear(wide, w, transpose=True)
        assert e.value.code == T.EXL3_ENOMEM


def test_binding_refuses(T, ctx):
    w = on_gpu(T, random_weight(128, 256, 2, 128, 291))
    we = on_gpu(T, random_weight(128, 256, 2, 128, 292, groups=2))
    x = torch.zeros(4, 256, dtype=BF, device=DEV)
    cut = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for bad in [lambda: ctx.linear(x.float(), w), lambda: ctx.linear(x[:, :128], w),
                lambda: ctx.linear(x.cpu(), w), lambda: ctx.linear(x[0], w),
                lambda: ctx.linear(x, we), lambda: ctx.grouped_linear(x, we, cut[:2]),
                lambda: ctx.grouped_linear(x, we, cut.long()),
                lambda: ctx.linear(x, w, out=torch.empty(4, 128, device=DEV)),
                lambda: ctx.linear(x, w, out=torch.empty(3, 128, dtype=BF, device=DEV))]:
        with pytest.raises(ValueError):
            bad()
    ad, *_ = adapters_of(T, 128, 256, 2, 8, FP, 293)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in [lambda: ctx.adapter_linear(x, w, ad, ids),
                lambda: ctx.adapter_linear(x.half(), w, ad, ids.long()),
                lambda: ctx.adapter_linear(x.half(), w, ad, ids[:3])]:
        with pytest.raises(ValueError):
            bad()


def test_timing_counts_a_product(T, ctx):
    w = on_gpu(T, random_weight(128, 256, 2, 128, 301))
    ctx.set_timing(True)
    ctx.linear(torch.zeros(4, 256, dtype=BF, device=DEV), w)
    ms, launches, tiles = ctx.read_timing("product")
    ctx.set_timing(False)
    assert launches == 1 and tiles == 8 * 16 and ms > 0


@pytest.mark.parametrize("pitch", [1 << 22, (1 << 22) + 8])
def test_rows_far_apart(T, ctx, pitch):
    """Rows of x so far apart that their offsets pass 2^27 bytes, and the pitch from which rows
    are packed before the product."""
    w = random_weight(128, 128, 2, 64, 311)
    x, x64 = rows_of(20, 128, FP, 312)
    far = torch.empty(19 * pitch + 128, dtype=FP, device=DEV)
    far = torch.as_strided(far, (20, 128), (pitch, 1))
    far.copy_(x)
    m = dense(w)
    y = ctx.linear(far, on_gpu(T, w), transpose=True)
    check(y, x64 @ m, spread_of(x64, m.T), inner_of(False, FP))
    y = ctx.linear(far, on_gpu(T, w))
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(False, FP))


@pytest.mark.parametrize("sizes", [[9, 0, 30, 17, 1], [8, 8, 8, 8], [33, 0, 0, 0, 0, 0, 0, 0]])
def test_few_rows_a_group_on_average(T, ctx, sizes):
    """Groups with more rows than the kernel takes at a time."""
    w = random_weight(192, 320, 2, 64, 321, groups=len(sizes))
    n = sum(sizes)
    x, x64 = rows_of(n, 320, BF, 322)
    cut = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    for repeat in range(2):          # the second call finds the first's counts at zero
        y = ctx.grouped_linear(x, on_gpu(T, w), torch.from_numpy(cut).to(DEV))
        for e in range(len(sizes)):
            if sizes[e]:
                m = dense(w, group=e)
                xe = x64[cut[e]:cut[e + 1]]
                check(y[cut[e]:cut[e + 1]], xe @ m.T, spread_of(xe, m), inner_of(True, BF))


@pytest.mark.parametrize("n", [1, 3, 4])
def test_one_launch_and_three_agree(T, ctx, n):
    """Rows that the smallest calls' kernel finishes itself, and the same among others."""
    w = random_weight(384, 2304, 2, 128, 331)
    x, x64 = rows_of(16, 2304, FP, 332)
    m = dense(w)
    g = on_gpu(T, w)
    want, spread = x64 @ m.T, spread_of(x64, m)
    check(ctx.linear(x[:n], g), want[:n], spread[:n], inner_of(True, FP))
    check(ctx.linear(x, g), want, spread, inner_of(True, FP))
