"""Products with coded weights over the ranges of their operands: level tables, channel scales and
adapters far from one, on both sides of the sizes at which the form changes."""
import numpy as np
import pytest
import torch

from product_reference import HALF, check, dense, inner_of, random_weight, spread_of
from test_gpu_products import (BF, DEV, FP, adapter_forward, adapters_of, ids_of, on_gpu,
                               rows_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    c = T.Context(0)
    yield c
    c.close()


def table_of(kind):
    """A caller's level table and the scale that takes it to a standard deviation near one."""
    r = np.random.Generator(np.random.PCG64(5))
    if kind == "sums":                  # the byte sums of mul1 before they are normalised
        h = (np.arange(65536, dtype=np.uint64) * 0x9E3779B1) & 0xFFFFFFFF
        t = sum((h >> s) & 255 for s in (0, 8, 16, 24)).astype(np.float64)
    else:
        t = r.standard_normal(65536) * kind
    return t.astype(np.float16), 1.0 / t.std()


# few rows; more than the general decoder's few rows take; and, transposed, the dense form always
@pytest.mark.parametrize("n,transpose", [(3, False), (64, False), (150, False), (3, True),
                                         (150, True)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", ["sums", 4000.0, 1e-3])
def test_level_tables_of_any_size(T, kind, dtype, n, transpose):
    table, scale = table_of(kind)
    w = random_weight(128, 256, 2, 128 if n == 3 else 64, 401)
    w["scale"] = np.float32(w["scale"] * scale)
    m = dense(w, table)
    m = m.T if transpose else m
    x, x64 = rows_of(n, m.shape[1], dtype, 402)
    with T.Context(0) as c:
        c.set_codebook(torch.from_numpy(table))
        y = c.linear(x, on_gpu(T, w), transpose=transpose)
        check(y, x64 @ m.T, spread_of(x64, m), inner_of(False, dtype))


# rows of a group up to which the levels are used themselves, and one more
THRESHOLD = [(512, False), (513, False), (256, True), (257, True)]


@pytest.mark.parametrize("n,transpose", THRESHOLD)
@pytest.mark.parametrize("size,std", [(1e-8, 500.0), (1e-5, 50.0), (1e5, 1e-3)])
def test_binary16_weights_of_any_size(T, ctx, size, std, n, transpose):
    w = random_weight(128, 192, 2, 64, 411)
    w["su"] = (w["su"] * (size / 0.02)).astype(np.float32)
    m = dense(w)
    m = m.T if transpose else m
    x, x64 = rows_of(n, m.shape[1], FP, 412, std)
    y = ctx.linear(x, on_gpu(T, w), transpose=transpose)
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(False, FP))


@pytest.mark.parametrize("n,transpose", THRESHOLD)
def test_binary16_channels_of_many_sizes(T, ctx, n, transpose):
    """Channels over 28 powers of two, and input channels over six.  Of a transposed product the
    input has large values where its channels are small."""
    r = np.random.Generator(np.random.PCG64(421))
    w = random_weight(128, 192, 3, 64, 422, dead=False)
    power = r.uniform(-20, -6, 128) if transpose else r.uniform(-26, 2, 128)
    w["su"] = (np.sign(w["su"]) * 2.0 ** power).astype(np.float32)
    w["sv"] = (w["sv"] * 2.0 ** r.uniform(-3, 3, 192)).astype(np.float32)
    m, inner = (dense(w).T, w["su"]) if transpose else (dense(w), w["sv"])
    inner = inner.astype(np.float64)
    z = r.standard_normal((n, m.shape[1])) * (2.0 ** (-8 - power) if transpose else 64.0)
    x = torch.from_numpy(z).to(FP)
    x64 = x.double().numpy()
    y = ctx.linear(x.to(DEV), on_gpu(T, w), transpose=transpose)
    # the transforms spread what the factors leave
    check(y, x64 @ m.T, spread_of(x64 * inner, m / inner), inner_of(False, FP))


@pytest.mark.parametrize("at", [0, 1, 2, 3, 126, 127])
@pytest.mark.parametrize("n,transpose", [(513, False), (257, True)])
def test_binary16_one_large_factor(T, ctx, n, transpose, at):
    """One factor of the contracted side far above the others, wherever it stands."""
    w = random_weight(128, 128, 2, 64, 426, dead=False)
    name = "su" if transpose else "sv"
    w[name][at] *= 2.0 ** 14
    m, inner = (dense(w).T, w["su"]) if transpose else (dense(w), w["sv"])
    inner = inner.astype(np.float64)
    x, x64 = rows_of(n, 128, FP, 427, 0.05)
    y = ctx.linear(x, on_gpu(T, w), transpose=transpose)
    check(y, x64 @ m.T, spread_of(x64 * inner, m / inner), inner_of(False, FP))


@pytest.mark.parametrize("per,transpose", [(513, False), (257, True)])
def test_binary16_groups_of_different_sizes(T, per, transpose):
    """Groups whose weights lie 40 powers of two apart, in batches of two of the dense form."""
    sizes = [1e-7, 1e5, 1.0, 1e-4, 1e2]
    w = random_weight(128, 192, 2, 64, 431, groups=5)
    w["su"] = (w["su"] * (np.array(sizes)[:, None] / 0.02)).astype(np.float32)
    n = 5 * per
    std = np.repeat([300.0, 1e-3, 1.0, 30.0, 0.1], per)[:, None]
    r = np.random.Generator(np.random.PCG64(432))
    x = torch.from_numpy(r.standard_normal((n, 128 if transpose else 192)) * std).to(FP)
    x64 = x.double().numpy()
    cut = torch.arange(6, dtype=torch.int32, device=DEV) * per
    with T.Context(0, scratch_bytes=2 * 128 * 192 * 2) as c:
        y = c.grouped_linear(x.to(DEV), on_gpu(T, w), cut, transpose=transpose)
        for e in range(5):
            m = dense(w, group=e)
            m = m.T if transpose else m
            at = slice(e * per, e * per + per)
            check(y[at], x64[at] @ m.T, spread_of(x64[at], m), inner_of(False, FP), "group %d" % e)


def check_subnormal(got, want, spread, inner, name):
    """check() for results that may lie in binary16's subnormal range, where a rounding is off by
    half a step of 2^-24 whatever the value: of every value, as there, and so of the whole."""
    off = np.abs(got.detach().double().cpu().numpy() - want)
    u, half_step = HALF[FP], 2.0 ** -25
    assert np.isfinite(off).all(), name
    bound = u * np.abs(want) * 1.001 + (8 / np.sqrt(3) * inner[0] + 2.0 ** -20) * spread + half_step
    assert (off <= bound).all(), "%s: %.3g times its bound" % (name, (off / bound).max())
    norm = np.linalg.norm(np.broadcast_to(spread, want.shape))
    assert np.linalg.norm(off) <= u * np.linalg.norm(want) + (inner[0] + 2.0 ** -20) * norm + \
        half_step * np.sqrt(want.size), name


# x, A, B and dy: alpha dy B far below binary16's normal range; alpha x A^T past its largest value
@pytest.mark.parametrize("n", [3, 40, 600])
@pytest.mark.parametrize("sx,sa,sb,sd", [(30.0, 1 / 16, 1e-3, 1e-5), (100.0, 60.0, 1e-4, 1e-4)])
def test_binary16_adapters_of_any_size(T, ctx, sx, sa, sb, sd, n):
    rows, cols, count, rank = 256, 256, 3, 12
    r = np.random.Generator(np.random.PCG64(441))
    w = random_weight(rows, cols, 2, 128, 442)
    A = torch.from_numpy(r.standard_normal((count, rank, cols)) * sa).to(FP)
    B = torch.from_numpy(r.standard_normal((count, rows, rank)) * sb).to(FP)
    al = torch.from_numpy((0.5 + r.random(count)).astype(np.float32))
    x, x64 = rows_of(n, cols, FP, 443, sx)
    dy, d64 = rows_of(n, rows, FP, 444, sd)
    ids = ids_of(n, count, 445)
    ad = T.Adapters(A.to(DEV), B.to(DEV), al.to(DEV))
    idt, g, m = torch.from_numpy(ids).to(DEV), on_gpu(T, w), dense(w)
    A, B, al = A.double().numpy(), B.double().numpy(), al.double().numpy()
    part, s = adapter_forward(x64, A, B, al, ids)
    y = ctx.adapter_linear(x, g, ad, idt)
    check_subnormal(y, x64 @ m.T + part, spread_of(x64, m) + s, inner_of(False, FP), "y")
    dx, dA, dB = ctx.adapter_linear_backward(dy, x, g, ad, idt)
    part, s = adapter_forward(d64, B.transpose(0, 2, 1), A.transpose(0, 2, 1), al, ids)
    check_subnormal(dx, d64 @ m + part, spread_of(d64, m.T) + s, inner_of(False, FP), "dx")
    for a in range(count):
        at = np.flatnonzero(ids == a)
        v, u = al[a] * (x64[at] @ A[a].T), al[a] * (d64[at] @ B[a])
        half = (HALF[FP], FP)
        check_subnormal(dA[a], u.T @ x64[at], np.sqrt((u ** 2).T @ x64[at] ** 2), half, "dA")
        check_subnormal(dB[a], d64[at].T @ v, np.sqrt((d64[at] ** 2).T @ v ** 2), half, "dB")


def test_binary16_rows_of_one_adapter_of_many_sizes(T, ctx):
    """Rows of one adapter, neighbours and far apart, over 20 powers of two: each row's part of y
    and dx is right by itself, the gradients' sums by the largest rows."""
    n, rows, cols, rank = 200, 128, 128, 8
    r = np.random.Generator(np.random.PCG64(451))
    w = random_weight(rows, cols, 2, 64, 452)
    ad, A, B, al = adapters_of(T, rows, cols, 1, rank, FP, 453)
    size = 2.0 ** r.uniform(-14, 6, n)[:, None]
    x = torch.from_numpy(r.standard_normal((n, cols)) * size).to(FP)
    dy = torch.from_numpy(r.standard_normal((n, rows)) * r.permutation(size)).to(FP)
    ids = np.zeros(n, np.int32)
    m, x64, d64 = dense(w), x.double().numpy(), dy.double().numpy()
    g, idt = on_gpu(T, w), torch.zeros(n, dtype=torch.int32, device=DEV)
    part, s = adapter_forward(x64, A, B, al, ids)
    check_subnormal(ctx.adapter_linear(x.to(DEV), g, ad, idt), x64 @ m.T + part,
                    spread_of(x64, m) + s, inner_of(False, FP), "y")
    dx, dA, dB = ctx.adapter_linear_backward(dy.to(DEV), x.to(DEV), g, ad, idt)
    part, s = adapter_forward(d64, B.transpose(0, 2, 1), A.transpose(0, 2, 1), al, ids)
    check_subnormal(dx, d64 @ m + part, spread_of(d64, m.T) + s, inner_of(False, FP), "dx")
    v, u = al[0] * (x64 @ A[0].T), al[0] * (d64 @ B[0])
    check_subnormal(dA[0], u.T @ x64, np.sqrt((u ** 2).T @ x64 ** 2), (HALF[FP], FP), "dA")
    check_subnormal(dB[0], d64.T @ v, np.sqrt((d64 ** 2).T @ v ** 2), (HALF[FP], FP), "dB")
