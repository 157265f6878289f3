"""Arguments of the products with coded weights that the binding and the C entries refuse without
a GPU, and the 64-bit reference of the GPU tests against a second route."""
import os

import numpy as np
import pytest
import torch

import oracle
from product_reference import dense, random_weight


@pytest.fixture(scope="module")
def lib():
    from trellis_coded_weight_amd import binding
    if not os.path.exists(binding.library_path()):
        pytest.skip("library not built")
    return binding.load_library()


def test_null_context_is_refused(lib):
    assert lib.exl3_linear(None, None, 0, None, 0, 0, 1, None, 0) == -1
    assert lib.exl3_grouped_linear(None, None, None, 0, None, 0, 0, 1, None, 0) == -1
    assert lib.exl3_adapter_linear(None, None, None, None, None, 0, 0, 1, None, 0) == -1
    assert lib.exl3_adapter_linear_backward(None, None, None, None, None, 0, None, 0, 0, 1, None,
                                            0, None, None) == -1


def test_holders_refuse_host_and_misshapen_tensors():
    from trellis_coded_weight_amd import Adapters, CodedWeight
    packed = torch.zeros(8, 8, 32, dtype=torch.int16)
    one = torch.ones(128)
    for args in [(packed, 2, 1.0, one, one), (packed[0], 2, 1.0, one, one),
                 (packed, 3, 1.0, one, one), (None, 2, 1.0, one, one)]:
        with pytest.raises(ValueError):
            CodedWeight(*args)
    with pytest.raises(ValueError):
        Adapters(torch.zeros(2, 4, 128), torch.zeros(2, 128, 4), torch.ones(2))
    with pytest.raises(ValueError):
        Adapters(torch.zeros(4, 128).bfloat16(), torch.zeros(128, 4).bfloat16(), torch.ones(1))


@pytest.mark.parametrize("had,K", [(64, 1), (128, 3)])
def test_dense_reference_is_the_oracles_inverse(had, K):
    w = random_weight(2 * had, had, K, had, 7)
    states = oracle.unpack_states(w["packed"].view(np.uint16).reshape(-1, 16 * K), K)
    lv = oracle.scaled_levels(oracle.mul1_levels_fp16(), w["scale"])
    m = oracle.unregularize(oracle.from_tiles(lv[states], 2 * had, had), w["su"], w["sv"], had)
    want = dense(w)
    # binary32 sums of had values, twice: a few tens of half steps of the largest
    assert np.abs(m - want).max() <= 64 * 2.0 ** -24 * np.abs(want).max()
