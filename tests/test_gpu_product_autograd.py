"""The differentiable functions over the products with coded weights, and the example that runs
them together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from product_reference import random_weight
from test_gpu_products import BF, DEV, FP, adapters_of, ids_of, on_gpu, rows_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.fixture(scope="module")
def ctx(T):
    c = T.Context(0)
    yield c
    c.close()


def test_linear_gradient_is_the_transposed_product(T, ctx):
    w = on_gpu(T, random_weight(128, 256, 2, 128, 1))
    x, _ = rows_of(30, 256, BF, 2)
    x = x.reshape(2, 15, 256).requires_grad_()
    y = T.coded_linear(ctx, x, w)
    assert y.shape == (2, 15, 128)
    assert torch.equal(y.detach(), ctx.linear(x.detach().reshape(30, 256), w).reshape(2, 15, 128))
    dy, _ = rows_of(30, 128, BF, 3)
    y.backward(dy.reshape(2, 15, 128))
    assert torch.equal(x.grad.reshape(30, 256), ctx.linear(dy, w, transpose=True))
    x.grad = None
    T.coded_linear(ctx, x, w).sum().backward()       # a gradient of one value, expanded
    ones = torch.ones(30, 128, dtype=BF, device=DEV)
    assert torch.equal(x.grad.reshape(30, 256), ctx.linear(ones, w, transpose=True))


def test_grouped_gradient(T, ctx):
    w = on_gpu(T, random_weight(128, 192, 2, 64, 11, groups=3))
    x, _ = rows_of(40, 192, FP, 12)
    x.requires_grad_()
    cut = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device=DEV)
    dy, _ = rows_of(40, 128, FP, 13)
    T.coded_grouped_linear(ctx, x, w, cut).backward(dy)
    assert torch.equal(x.grad, ctx.grouped_linear(dy, w, cut, transpose=True))


@pytest.mark.parametrize("wants", [(True, True, True), (False, True, True), (True, False, False),
                                   (False, True, False)])
def test_adapter_gradients(T, ctx, wants):
    w = on_gpu(T, random_weight(128, 256, 3, 128, 21))
    ad, *_ = adapters_of(T, 128, 256, 3, 8, BF, 22)
    x, _ = rows_of(50, 256, BF, 23)
    dy, _ = rows_of(50, 128, BF, 24)
    ids = torch.from_numpy(ids_of(50, 3, 25)).to(DEV)
    want = ctx.adapter_linear_backward(dy, x, w, ad, ids)
    args = [t.clone().requires_grad_(g) for t, g in zip((x, ad.A, ad.B), wants)]
    y = T.coded_adapter_linear(ctx, args[0], w, args[1], args[2], ad.alpha, ids)
    assert torch.equal(y.detach(), ctx.adapter_linear(x, w, ad, ids))
    y.backward(dy)
    for a, g, e in zip(args, wants, want):
        assert (a.grad is None) if not g else torch.equal(a.grad, e)


def test_example_layer():
    spec = importlib.util.spec_from_file_location(
        "coded_layer", os.path.join(ROOT, "examples", "coded_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, same, losses = m.main(["--rows", "256", "--experts", "4", "--tokens", "200", "--bits",
                                "4", "--steps", "10"])
    # two matrices of K = 4 codes, each about 0.09 of its norm off
    assert 0.02 < off < 0.3
    # one token may go to another expert than in the prompt only on a tie of the router
    assert same < 0.05
    assert losses[-1] < losses[0] and np.isfinite(losses).all()
