"""What the differentiable products keep between forward and backward, and what they refuse to
differentiate after it has changed."""
import numpy as np
import pytest
import torch

from product_reference import random_weight
from test_gpu_products import BF, DEV, adapters_of, ids_of, on_gpu, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


def _call(T, c, op, x, w, we, ad, ids, cut):
    if op == "linear":
        return T.coded_linear(c, x, w)
    if op == "grouped":
        return T.coded_grouped_linear(c, x, we, cut)
    return T.coded_adapter_linear(c, x, w, ad.A, ad.B, ad.alpha, ids)


def _setup(T, op):
    w = on_gpu(T, random_weight(128, 256, 2, 128, 501))
    we = on_gpu(T, random_weight(128, 256, 2, 128, 502, groups=2))
    ad, *_ = adapters_of(T, 128, 256, 2, 8, BF, 503)
    x, _ = rows_of(12, 256, BF, 504)
    dy, _ = rows_of(12, 128, BF, 505)
    ids = torch.from_numpy(ids_of(12, 2, 506)).to(DEV)
    cut = torch.tensor([0, 5, 12], dtype=torch.int32, device=DEV)
    return w, we, ad, ids, cut, x.requires_grad_(), dy


ORDER = np.arange(256)[::-1].copy()
TABLE = torch.linspace(-2, 2, 65536).half()


@pytest.mark.parametrize("op", ["linear", "grouped", "adapters"])
@pytest.mark.parametrize("change,back", [
    (lambda c: c.set_codebook_kind("mcg"), lambda c: c.set_codebook_kind("mul1")),
    (lambda c: c.set_codebook(TABLE), lambda c: c.set_codebook(None)),
    (lambda c: c.set_tile_order(ORDER), lambda c: c.set_tile_order(None))])
def test_a_gradient_under_other_levels_is_refused(T, op, change, back):
    """The levels and the order are the context's: with others in place the gradient would be
    another matrix's.  Set as they were, they serve."""
    w, we, ad, ids, cut, x, dy = _setup(T, op)
    with T.Context(0) as c:
        y = _call(T, c, op, x, w, we, ad, ids, cut)
        y.backward(dy, retain_graph=True)
        want, x.grad = x.grad, None
        change(c)
        with pytest.raises(RuntimeError, match="codebook"):
            y.backward(dy, retain_graph=True)
        assert x.grad is None
        back(c)
        y.backward(dy)
        assert torch.equal(x.grad, want)
        # the same under the other levels throughout
        x.grad = None
        change(c)
        _call(T, c, op, x, w, we, ad, ids, cut).backward(dy)
        assert x.grad is not None and not torch.equal(x.grad, want)
        torch.cuda.synchronize()


def test_levels_set_again_are_the_same_levels(T):
    w, we, ad, ids, cut, x, dy = _setup(T, "linear")
    with T.Context(0) as c:
        c.set_tile_order(np.arange(256))
        assert c._decoder() == ("mul1", None)
        c.set_codebook(TABLE)
        c.set_tile_order(ORDER)
        y = T.coded_linear(c, x, w)
        c.set_codebook_kind("3inst")
        c.set_tile_order(None)
        c.set_codebook(TABLE.clone())
        c.set_tile_order(list(ORDER))
        y.backward(dy)
        assert x.grad is not None
        torch.cuda.synchronize()


@pytest.mark.parametrize("op", ["linear", "grouped", "adapters"])
@pytest.mark.parametrize("name", ["packed", "scale", "su", "sv"])
def test_a_weight_changed_in_place_is_refused(T, op, name):
    """As torch refuses any tensor that a backward pass needs and that has changed since."""
    w, we, ad, ids, cut, x, dy = _setup(T, op)
    with T.Context(0) as c:
        y = _call(T, c, op, x, w, we, ad, ids, cut)
        getattr(we if op == "grouped" else w, name).neg_()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward(dy)
        torch.cuda.synchronize()


def test_alpha_has_no_gradient(T):
    """Refused, where a silent None would leave it untrained."""
    w, we, ad, ids, cut, x, dy = _setup(T, "adapters")
    with T.Context(0) as c:
        alpha = ad.alpha.clone().requires_grad_()
        with pytest.raises(ValueError, match="alpha"):
            T.coded_adapter_linear(c, x, w, ad.A, ad.B, alpha, ids)
        with torch.no_grad():
            y = T.coded_adapter_linear(c, x, w, ad.A, ad.B, alpha, ids)
        assert torch.equal(y, T.coded_adapter_linear(c, x, w, ad.A, ad.B, alpha.detach(), ids))
        torch.cuda.synchronize()
