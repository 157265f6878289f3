"""Reference of the operators in 8-bit blocks: the writing of blocks in binary32 on the CPU (each
step one IEEE operation, so the kernels have to agree bit for bit), everything else in 64 bits."""
import torch

E4M3 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half the smallest step


def blocks(width):
    return -(-width // 128)


def to_blocks(v, rows=1):
    """v [R, C] float32 on the CPU -> (codes e4m3 [R, C], scales [R / rows, C / 128])."""
    R, C = v.shape
    p = torch.zeros(-(-R // rows) * rows, 128 * blocks(C))
    p[:R, :C] = v
    p = p.reshape(p.shape[0] // rows, rows, blocks(C), 128)
    big = p.abs().amax(dim=(1, 3))
    scale = torch.clamp(big / 448.0, min=2.0 ** -126)
    scale = torch.where(torch.isfinite(big), scale, float("nan"))
    q = (p / scale[:, None, :, None]).to(E4M3)
    return q.reshape(-1, 128 * blocks(C))[:R, :C].contiguous(), scale


def from_blocks(q, scale, rows=1):
    s = scale.double().repeat_interleave(128, dim=1).repeat_interleave(rows, dim=0)
    return q.double() * s[:q.shape[0], :q.shape[1]]


def rows_of(n, cols, dtype, seed, spread=1.0, device="cuda", pitch=None, at=0):
    """(rows on the device, of any pitch and start, the same on the CPU)."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(n, cols, generator=g) * spread
    v = (v * torch.where(torch.rand(cols, generator=g) < 0.02, 12.0, 1.0)).to(dtype)
    flat = torch.full((at + max(n, 1) * (pitch or cols),), 7.0, dtype=dtype)
    dev = flat.to(device)[at:].as_strided((n, cols), (pitch or cols, 1))
    dev.copy_(v)
    return dev, v


def norm(s, gain, eps):
    """(y, r) in 64 bits from s [n, cols]."""
    s = s.double()
    r = 1.0 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + eps)
    return s * r * gain.double(), r


def product(x, w):
    """x [n, k] times w [m, k] in 64 bits and the sum of magnitudes."""
    x, w = x.double(), w.double()
    return x @ w.t(), x.abs() @ w.abs().t()
