"""Capturing products with coded weights on another stream than the calls before used."""
import pytest
import torch

from product_reference import random_weight
from test_gpu_products import BF, rows_of, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import trellis_coded_weight_amd as T
    return T


@pytest.mark.parametrize("first", ["side", "default"])
@pytest.mark.parametrize("n", [2, 40, 600])
def test_a_capture_on_torchs_own_stream(T, n, first):
    """Warmed up on one stream, captured on the one that torch takes, used on the first again."""
    w = on_gpu(T, random_weight(256, 384, 2, 128, 701))
    x, _ = rows_of(n, 384, BF, 702)
    with T.Context(0) as c, T.Context(0) as other:
        if first == "side":
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                c.linear(x, w)
            torch.cuda.current_stream().wait_stream(side)
        else:
            c.linear(x, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = c.linear(x, w)
        for seed in range(3):
            xn, _ = rows_of(n, 384, BF, 710 + seed)
            want = other.linear(xn, w)
            x.copy_(xn)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            assert torch.equal(c.linear(xn, w), want)
        torch.cuda.synchronize()
        del graph


def test_a_capture_with_work_left_is_refused_and_goes_on(T):
    w = on_gpu(T, random_weight(4096, 4096, 2, 128, 703))
    x, _ = rows_of(4096, 4096, BF, 704)
    with T.Context(0) as c:
        for _ in range(3):
            c.linear(x, w)
        torch.cuda.synchronize()
        graph, side, out = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.zeros(4, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(100):                       # tens of milliseconds of work
                c.linear(x, w)
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            graph.capture_begin(capture_error_mode="relaxed")
            out += 1
            with pytest.raises(T.Exl3Error) as e:
                c.linear(x, w)
            graph.capture_end()
        torch.cuda.synchronize()
        assert e.value.code == T.EXL3_EINVAL and "captur" in e.value.msg
        graph.replay()
        torch.cuda.synchronize()
        assert (out == 1).all()
        assert torch.isfinite(c.linear(x, w)).all()
        torch.cuda.synchronize()
        del graph
