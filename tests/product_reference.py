"""Products with coded weights in 64 bits on the CPU, from the oracle's container reader and
level tables, and the bounds their tests use (shared by the CPU and GPU tests)."""
import numpy as np
import scipy.linalg
import torch

import oracle

# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def levels(codebook):
    table = {"mul1": oracle.mul1_levels_fp16, "mcg": oracle.mcg_levels_fp16,
             "3inst": oracle.inst3_levels_fp16}
    return table[codebook]() if isinstance(codebook, str) else codebook


def random_weight(rows, cols, K, had, seed, groups=None, dead=True):
    """Container words, scale, su (folded channel scales, one dead channel) and sv as numpy
    arrays; every bit string is a container."""
    r = np.random.Generator(np.random.PCG64(seed))
    lead = () if groups is None else (groups,)
    packed = r.integers(-32768, 32768, lead + (rows // 16, cols // 16, 16 * K)).astype(np.int16)
    su = ((2 * r.integers(0, 2, lead + (rows,)) - 1) *
          0.02 * np.exp(0.3 * r.standard_normal(lead + (rows,)))).astype(np.float32)
    if dead:
        su[..., 5] = 0.0
    sv = (2 * r.integers(0, 2, lead + (cols,)) - 1).astype(np.float32)
    scale = (0.8 + 0.4 * r.random(lead)).astype(np.float32)
    return {"packed": packed, "scale": scale, "su": su, "sv": sv, "K": K, "had": had,
            "groups": groups}


def dense(w, codebook="mul1", order=None, group=None):
    """W in float64."""
    at = (lambda a: a) if group is None else (lambda a: a[group])
    packed, K, hb = at(w["packed"]), w["K"], w["had"]
    rows, cols = 16 * packed.shape[0], 16 * packed.shape[1]
    states = oracle.unpack_states(packed.view(np.uint16).reshape(-1, 16 * K), K)
    lv = np.asarray(levels(codebook)).view(np.float16).astype(np.float64)
    m = oracle.from_tiles(lv[states], rows, cols, order).astype(np.float64)
    h = scipy.linalg.hadamard(hb) / np.sqrt(hb)
    m = (m.reshape(-1, hb) @ h).reshape(rows, cols)
    m = np.einsum("ij,bjc->bic", h, m.reshape(-1, hb, cols)).reshape(rows, cols)
    return m * float(at(w["scale"])) * at(w["su"]).astype(np.float64)[:, None] * \
        at(w["sv"]).astype(np.float64)[None, :]


def check(got, want, spread, inner, name=""):
    """got against the 64-bit want.

    Two roundings enter: the output's, half a step of its type of every value, and those
    inside (`inner`: the sum of the half steps of the operands that are rounded), independent
    over the terms of a sum.  A sum of terms each off by at most inner / sqrt(3) (the rms of a
    rounding uniform in its half step) of themselves is off by that much of `spread`, the
    root of the sum of the terms' squares; eight times that bounds every value (normal tails),
    and once the half steps bound the whole in 2-norm."""
    got = got.detach().double().cpu().numpy()
    u = HALF[torch.bfloat16] if inner[1] is torch.bfloat16 else HALF[torch.float16]
    off = np.abs(got - want)
    # 2^-20 of the spread: the binary32 sums
    bound = u * np.abs(want) * 1.001 + (8 / np.sqrt(3) * inner[0] + 2.0 ** -20) * spread + 2.0 ** -25
    assert np.isfinite(got).all(), name
    worst = float((off / bound).max()) if off.size else 0.0
    assert worst <= 1.0, "%s: a value is %.3g times its bound off" % (name, worst)
    norm = np.linalg.norm(np.broadcast_to(spread, want.shape)) if off.size else 0.0
    total = np.linalg.norm(off)
    assert total <= u * np.linalg.norm(want) + (inner[0] + 2.0 ** -20) * norm + 1e-6 * norm + 1e-20, \
        "%s: off by %.3g of the norm" % (name, total / max(norm, 1e-300))


def spread_of(x, w):
    """For y = x w^T with both sides spread evenly by the transforms: |x_t| |w_r| / sqrt(k)."""
    return np.linalg.norm(x, axis=1)[:, None] * np.linalg.norm(w, axis=1)[None, :] / \
        np.sqrt(x.shape[1])


def inner_of(few, dtype):
    """Half steps inside a product: few rows, x' in binary16; many, the half-transformed levels
    in binary16 and the weights in the activations' type."""
    return (HALF[torch.float16] if few else HALF[torch.float16] + HALF[dtype], dtype)
