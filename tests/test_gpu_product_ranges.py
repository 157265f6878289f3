"""Products with coded weights over the ranges of their operands: level tables, channel scales and
adapters far from one, on both sides of the sizes at which the form changes."""
import numpy as np
import pytest
import torch

from product_reference import check, dense, inner_of, random_weight, spread_of
from test_gpu_products import BF, DEV, FP, on_gpu, rows_of

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
