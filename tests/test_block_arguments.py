"""Arguments of the operators in 8-bit blocks that the binding and the C entries refuse without a
GPU, and the GPU tests' reference of writing blocks against a second route."""
import os

import pytest
import torch

from block_reference import E4M3, from_blocks, to_blocks


@pytest.fixture(scope="module")
def lib():
    from trellis_coded_weight_amd import binding
    if not os.path.exists(binding.library_path()):
        pytest.skip("library not built")
    return binding.load_library()


def test_null_context_is_refused(lib):
    assert lib.exl3_block_quantize(None, None, 0, 0, 1, 1, None) == -1
    assert lib.exl3_block_quantize_weight(None, None, 0, 1, 1, 0, None, 0, None) == -1
    assert lib.exl3_rms_norm(None, None, 0, None, 0, None, 0, 0.0, 0, 1, 1, None, 0, None, None,
                             0) == -1
    assert lib.exl3_rms_norm_backward(None, None, 0, None, 0, None, 0, None, 0, 0.0, 0, 1, 1, None,
                                      0, None) == -1
    assert lib.exl3_block_linear(None, None, 0, None, 0, None, 0, 1, None, 0) == -1
    assert lib.exl3_block_grouped_linear(None, None, None, 0, None, 0, None, 0, 1, None, 0) == -1


def test_holders_refuse_host_and_misshapen_tensors():
    from trellis_coded_weight_amd import BlockRows, BlockWeight
    q = torch.zeros(128, 256).to(E4M3)
    for args in [(q, torch.ones(1, 2)), (q.float(), torch.ones(1, 2)), (None, None), (q[0], q)]:
        with pytest.raises(ValueError):
            BlockWeight(*args)
        with pytest.raises(ValueError):
            BlockRows(*args)


def test_reference_rounds_to_the_nearest_code():
    """Against a search over all 256 codes in 64 bits."""
    g = torch.Generator().manual_seed(1)
    v = torch.randn(5, 300, generator=g).bfloat16().float()
    v[1, :128] = 0
    q, scale = to_blocks(v)
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).double()
    codes = codes[torch.isfinite(codes)]
    s = scale.double().repeat_interleave(128, 1)[:, :300]
    best = (codes[None, None] - (v.double() / s)[..., None]).abs().min(dim=2).values
    got = (q.double() - v.double() / s).abs()
    # the quotient's own rounding may decide what lies within it of a tie
    assert (got <= best + 2.0 ** -23 * 448).all()
    assert torch.equal(from_blocks(q, scale), q.double() * s)


def test_a_residual_of_another_shape_is_refused():
    """Also one of as many rows, which flattening would pair with others."""
    from trellis_coded_weight_amd import rms_norm
    x, gain = torch.zeros(2, 3, 8).bfloat16(), torch.ones(8)
    for shape in [(3, 2, 8), (6, 8), (1, 3, 8), (2, 3, 1), (8,)]:
        with pytest.raises(ValueError, match="residual must have shape"):
            rms_norm(None, x, gain, residual=torch.zeros(shape).bfloat16())
