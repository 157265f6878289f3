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
