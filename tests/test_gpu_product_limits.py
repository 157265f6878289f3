"""Products with coded weights at the limits of their arguments, and forms that only certain
alignments, sizes or scratch bounds reach."""
import numpy as np
import pytest
import torch

from product_reference import HALF, check, dense, inner_of, random_weight, spread_of
from test_gpu_products import (BF, DEV, FP, adapter_forward, adapters_of, ids_of, on_gpu, rows_of)

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


def unaligned(T, w):
    """The weight with words that start on 8 bytes, which the tiles' kernel does not take."""
    g = on_gpu(T, w)
    flat = torch.zeros(g.packed.numel() + 4, dtype=torch.int16, device=DEV)
    flat[4:] = g.packed.reshape(-1)
    h = T.CodedWeight(flat[4:].view(g.packed.shape), w["K"], g.scale, g.su, g.sv,
                      had_block=w["had"])
    assert h.packed.data_ptr() % 16 == 8
    return h


def cut_of(sizes, first=0):
    cut = first + np.concatenate([[0], np.cumsum(sizes)])
    return cut, torch.from_numpy(cut.astype(np.int32)).to(DEV)


def check_groups(y, x64, w, cut, transpose, dtype):
    for e in range(len(cut) - 1):
        if cut[e + 1] > cut[e]:
            m = dense(w, group=e)
            m = m.T if transpose else m
            xe = x64[cut[e]:cut[e + 1]]
            check(y[cut[e]:cut[e + 1]], xe @ m.T, spread_of(xe, m), inner_of(False, dtype),
                  "group %d" % e)


# ---- dense weights of groups ----
# more than 64 rows a group on average, so that also x W^T takes the dense form
@pytest.mark.parametrize("K,dtype", [(2, BF), (2, FP), (3, BF), (5, FP), (8, BF)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 3])
def test_dense_groups_in_batches(T, K, dtype, transpose, batch):
    """As many groups at a time as the scratch bound holds: empty groups at the batches' ends,
    rows before the first group and after the last."""
    sizes = [130, 0, 0, 301, 64, 0, 70]
    w = random_weight(128, 192, K, 64, 601 + K, groups=7)
    cut, at = cut_of(sizes, 5)
    n = int(cut[-1]) + 9
    x, x64 = rows_of(n, 128 if transpose else 192, dtype, 602)
    with T.Context(0, scratch_bytes=batch * 128 * 192 * 2) as c:
        y = torch.full((n, 192 if transpose else 128), 7.0, dtype=dtype, device=DEV)
        c.grouped_linear(x, unaligned(T, w), at, transpose=transpose, out=y)
        assert (y[:5] == 0).all() and (y[int(cut[-1]):] == 0).all()
        check_groups(y, x64, w, cut, transpose, dtype)
        torch.cuda.synchronize()


@pytest.mark.parametrize("K", [5, 6, 7, 8])
@pytest.mark.parametrize("per", [3, 12, 40, 90])
@pytest.mark.parametrize("transpose", [False, True])
def test_general_decoder_of_groups(T, ctx, K, per, transpose):
    w = random_weight(192, 128, K, 64, 611 + K, groups=3)
    cut, at = cut_of([per, 0, per + 1], 2)
    n = int(cut[-1]) + 3
    x, x64 = rows_of(n, 192 if transpose else 128, FP, 612)
    y = ctx.grouped_linear(x, on_gpu(T, w), at, transpose=transpose)
    assert (y[:2] == 0).all() and (y[int(cut[-1]):] == 0).all()
    check_groups(y, x64, w, cut, transpose, FP)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_one_launch_with_rows_of_no_group(T, ctx, dtype):
    """Few enough rows that the first kernel writes y itself, the rows of no group included."""
    w = random_weight(128, 256, 2, 128, 621, groups=3)
    cut, at = cut_of([2, 0, 4], 3)
    x, x64 = rows_of(12, 256, dtype, 622)
    for repeat in range(2):
        y = torch.full((12, 128), 7.0, dtype=dtype, device=DEV)
        ctx.grouped_linear(x, on_gpu(T, w), at, out=y)
        assert (y[:3] == 0).all() and (y[9:] == 0).all()
        check_groups(y, x64, w, cut, False, dtype)


# ---- long rows ----
@pytest.mark.parametrize("cols,had", [(4096 + 128, 128), (16384 + 64, 64), (16384 + 4096 + 128, 128)])
@pytest.mark.parametrize("n", [2, 9, 40])
def test_long_rows(T, ctx, cols, had, n):
    """Rows of x that a workgroup transforms in several rounds, and past 16,384 columns twice."""
    w = random_weight(128, cols, 2, had, 631)
    m = dense(w)
    x, x64 = rows_of(n, cols, BF, 632)
    check(ctx.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(True, BF))
    w = random_weight(cols, 128, 2, had, 633)
    m = dense(w).T
    x, x64 = rows_of(n, cols, FP, 634)
    y = ctx.linear(x, on_gpu(T, w), transpose=True)
    check(y, x64 @ m.T, spread_of(x64, m), inner_of(True, FP))


# ---- the decoded forms by their own bound ----
@pytest.mark.parametrize("n,rows,cols,K,had,codebook", [
    (1, 256, 1152, 1, 128, "mul1"), (15, 384, 2176, 4, 128, "mcg"), (17, 640, 256, 3, 128, "3inst"),
    (40, 192, 320, 2, 64, "mul1"), (65, 128, 1152, 3, 128, "mul1"), (300, 640, 576, 2, 64, "mcg"),
    (512, 128, 256, 4, 128, "mul1")])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decoded_forms_round_the_activations_only(T, n, rows, cols, K, had, codebook, dtype):
    w = random_weight(rows, cols, K, had, 641 + n)
    m = dense(w, codebook)
    x, x64 = rows_of(n, cols, dtype, 642)
    with T.Context(0) as c:
        c.set_codebook_kind(codebook)
        check(c.linear(x, on_gpu(T, w)), x64 @ m.T, spread_of(x64, m), inner_of(True, dtype))
        if n <= 256:
            x, x64 = rows_of(n, rows, dtype, 643)
            y = c.linear(x, on_gpu(T, w), transpose=True)
            check(y, x64 @ m, spread_of(x64, m.T), inner_of(True, dtype))
        torch.cuda.synchronize()


# ---- many adapters ----
def test_many_adapters(T, ctx):
    """Past half of the largest count, most of them without rows."""
    n, count = 150, 40000
    w = random_weight(128, 64, 2, 64, 651)
    ad, A, B, al = adapters_of(T, 128, 64, count, 1, BF, 652)
    r = np.random.Generator(np.random.PCG64(653))
    ids = r.integers(0, count, n).astype(np.int32)
    ids[:3] = [0, count - 1, count - 1]
    idt, g, m = torch.from_numpy(ids).to(DEV), on_gpu(T, w), dense(w)
    x, x64 = rows_of(n, 64, BF, 654)
    dy, d64 = rows_of(n, 128, BF, 655, 0.05)
    part, s = adapter_forward(x64, A, B, al, ids)
    y = ctx.adapter_linear(x, g, ad, idt)
    check(y, x64 @ m.T + part, spread_of(x64, m) + s, inner_of(False, BF))
    dx, dA, dB = ctx.adapter_linear_backward(dy, x, g, ad, idt)
    part, s = adapter_forward(d64, B.transpose(0, 2, 1), A.transpose(0, 2, 1), al, ids)
    check(dx, d64 @ m + part, spread_of(d64, m.T) + s, inner_of(False, BF), "dx")
    for a in np.unique(ids):
        at = np.flatnonzero(ids == a)
        v, u = al[a] * (x64[at] @ A[a].T), al[a] * (d64[at] @ B[a])
        half = (HALF[BF], BF)
        check(dA[a], u.T @ x64[at], np.sqrt((u ** 2).T @ x64[at] ** 2), half, "dA")
        check(dB[a], d64[at].T @ v, np.sqrt((d64[at] ** 2).T @ v ** 2), half, "dB")
    rest = torch.ones(count, dtype=torch.bool, device=DEV)
    rest[idt.long()] = False
    assert (dA[rest] == 0).all() and (dB[rest] == 0).all()


# ---- workspace ----
def test_a_gradient_of_the_activations_alone_needs_little_workspace(T):
    """dx takes the two small products and W, nothing for the matrices' gradients: their sums
    alone would be 4 parts of 32 adapters, 268 MB for each matrix."""
    rows = cols = 8192
    g = torch.zeros(rows // 16, cols // 16, 32, dtype=torch.int16, device=DEV)
    w = T.CodedWeight(g, 2, 1.0, torch.ones(rows, device=DEV), torch.ones(cols, device=DEV))
    A = torch.zeros(32, 64, cols, dtype=BF, device=DEV)
    B = torch.zeros(32, rows, 64, dtype=BF, device=DEV)
    ad = T.Adapters(A, B, torch.ones(32, device=DEV))
    n = 512
    x, dy = torch.zeros(n, cols, dtype=BF, device=DEV), torch.zeros(n, rows, dtype=BF, device=DEV)
    ids = torch.zeros(n, dtype=torch.int32, device=DEV)
    with T.Context(0) as c:
        c.linear(dy[:1], w)                                 # what any call brings along
        keep = torch.empty(n, cols, dtype=BF, device=DEV)   # dx comes from torch's pool
        del keep
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        dx, dA, dB = c.adapter_linear_backward(dy, x, w, ad, ids, want_adapters=False)
        torch.cuda.synchronize()
        took = free - torch.cuda.mem_get_info()[0]
        assert dA is None and dB is None and (dx == 0).all()
        # W 134 MB, A and B transposed 34 MB each
        assert took < 260e6, took


# ---- offsets that no program should pass ----
def test_offsets_that_claim_rows_over_and_over(T, ctx):
    """Every other group claims all rows, 2^31 tiles and more between them: rows are unspecified,
    but nothing is written beside them."""
    groups, n = 65535, 1 << 22
    packed = torch.zeros(groups * 4 * 20 * 16 + 4, dtype=torch.int16, device=DEV)
    w = T.CodedWeight(packed[4:].view(groups, 4, 20, 16), 1, torch.ones(groups, device=DEV),
                      torch.ones(groups, 64, device=DEV), torch.ones(groups, 320, device=DEV),
                      had_block=64)
    at = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    at[1::2] = n
    x = torch.zeros(n, 64, dtype=BF, device=DEV)
    flat = torch.full((n * 320 + 2048,), 3.0, dtype=BF, device=DEV)
    ctx.grouped_linear(x, w, at, transpose=True, out=flat[1024:-1024].view(n, 320))
    torch.cuda.synchronize()
    assert (flat[:1024] == 3.0).all() and (flat[-1024:] == 3.0).all()


# ---- the most rows ----
def test_the_most_rows(T, ctx):
    """2^24 rows: the kernels with a workgroup a row have more lanes than one launch takes."""
    groups, n = 32768, 1 << 24
    w = random_weight(64, 64, 1, 64, 661, groups=4)
    big = {k: (np.concatenate([v] * (groups // 4)) if isinstance(v, np.ndarray) else v)
           for k, v in w.items()}
    g = on_gpu(T, big)
    x, x64 = rows_of(2048, 64, BF, 662)
    at = torch.arange(groups + 1, dtype=torch.int32, device=DEV) * (n // groups)
    y = ctx.grouped_linear(x.repeat(n // 2048, 1), g, at)
    first = y[:2048]
    for e in range(4):
        m, xe = dense(w, group=e), x64[512 * e:512 * e + 512]
        check(first[512 * e:512 * e + 512], xe @ m.T, spread_of(xe, m), inner_of(True, BF))
    assert (y.view(n // 2048, 2048, 64) == first).all()
