"""Measured cases of the products with trellis-coded weights.

Three operators, each on a matrix W [rows, cols] held as a container of K-bit trellis codes,
a scale and two sign-and-scale vectors, W = diag(su) H_l (scale * level[state]) H_r diag(sv)
(H: blockwise normalised Sylvester Hadamard):

  linear     y = x W^T, and its input gradient dx = dy W
  grouped    the same with a weight per expert, over rows sorted by expert (ragged groups)
  adapters   y = x W^T + alpha_a (x A_a^T) B_a^T with an adapter a per row (or none), and its
             backward pass: dx, dA, dB

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true,
through the package's entry points.  ``exact`` computes them in 64 bits by another route (the
codes' bits unfolded one by one, and the transforms applied to the activations).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, direction, n, rows, cols, K, dtype, had=128, codebook="mul1", experts=1,
          adapters=0, rank=0):
    c = {"op": op, "direction": direction, "n": n, "rows": rows, "cols": cols, "K": K,
         "dtype": dtype, "had": had, "codebook": codebook, "experts": experts,
         "adapters": adapters, "rank": rank}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence being generated, a key or value projection: the smallest call
        _case("linear 1x1024x4096 K2", "linear", "forward", 1, 1024, 4096, 2, "bf16"),
        # one sequence being generated, an MLP projection
        _case("linear 1x12288x4096 K4", "linear", "forward", 1, 12288, 4096, 4, "fp16"),
        # a batch of sequences being generated, an MLP's second projection
        _case("linear 24x4096x12288 K3", "linear", "forward", 24, 4096, 12288, 3, "bf16"),
        # a short prompt of an odd length, the additive codebook
        _case("linear 333x4096x4096 K2", "linear", "forward", 333, 4096, 4096, 2, "fp16",
              codebook="3inst"),
        # a long prompt through an MLP projection: the largest call
        _case("linear 4096x12288x4096 K2", "linear", "forward", 4096, 12288, 4096, 2, "bf16"),
        # a training step through a frozen coded projection
        _case("linear grad 2000x4096x4096 K4", "linear", "backward", 2000, 4096, 4096, 4, "bf16"),
        # eight tokens with eight experts each: few rows an expert, some experts none
        _case("grouped 64x1408x2048 E64 K2", "grouped", "forward", 64, 1408, 2048, 2, "bf16",
              experts=64),
        # a prompt through the same experts, groups of uneven sizes
        _case("grouped 8200x1408x2048 E64 K3", "grouped", "forward", 8200, 1408, 2048, 3, "bf16",
              experts=64),
        # a training step through an expert layer's second projection, 64-point transforms
        _case("grouped grad 4001x2048x1408 E16", "grouped", "backward", 4001, 2048, 1408, 2,
              "fp16", had=64, experts=16),
        # 32 requests being generated, each with an adapter of its own
        _case("adapters 32x4096x4096 r16", "adapters", "forward", 32, 4096, 4096, 3, "bf16",
              adapters=32, rank=16),
        # prompts of a few requests in one batch, wide adapters
        _case("adapters 1500x4096x4096 r64", "adapters", "forward", 1500, 4096, 4096, 2, "fp16",
              adapters=8, rank=64),
        # a training step of adapters on a frozen coded projection
        _case("adapters grad 2048x4096x4096 r16", "adapters", "backward", 2048, 4096, 4096, 2,
              "bf16", adapters=4, rank=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "grouped", "adapters"])
    direction = rng.choice(["forward", "forward", "backward"])
    had = rng.choice([128, 128, 64])
    K = rng.choice([1, 2, 2, 3, 4])
    dtype = rng.choice(["bf16", "fp16"])
    codebook = rng.choice(["mul1", "mul1", "mcg", "3inst"])
    n = _log_int(rng, 1, 4096) if direction == "forward" else _log_int(rng, 100, 4096)
    if op == "grouped":
        side = [had * rng.randint(512 // had, 2048 // had) for _ in range(2)]
        return _case(None, op, direction, n, side[0], side[1], K, dtype, had, codebook,
                     experts=rng.randint(4, 64))
    side = [had * _log_int(rng, 512 // had, 8192 // had) for _ in range(2)]
    if op == "linear":
        return _case(None, op, direction, n, side[0], side[1], K, dtype, had, codebook)
    return _case(None, op, direction, n, side[0], side[1], K, dtype, had, codebook,
                 adapters=rng.randint(1, 32), rank=rng.choice([4, 8, 12, 16, 32, 64]))


def work(case):
    c = case
    n, R, C = c["n"], c["rows"], c["cols"]
    E = c["experts"]
    # experts that some row goes to, each row's expert drawn from _expert_share
    used = float((1 - (1 - _expert_share(E)) ** n).sum()) if E > 1 else 1.0
    weight = used * (R * C * c["K"] / 8 + 4 * (R + C + 1))
    b = weight + 2 * n * (R + C)
    f = 2.0 * n * R * C
    if c["op"] == "adapters":
        r, m = c["rank"], min(c["adapters"], n)
        b += 2 * m * r * (R + C) + 4 * n
        f += 2.0 * n * r * (R + C)
        if c["direction"] == "backward":
            # x as well as dy is read, dA and dB are written, the two products that give them
            # and the forward's first one again
            b += 2 * n * C + 2 * c["adapters"] * r * (R + C)
            f += 2.0 * n * r * (R + 2 * C)
    return {"bytes": b, "flops": f}


def _expert_share(E):
    """How often each expert is chosen: the busiest about six times as often as the median."""
    p = 1.0 / (1.0 + np.arange(E)) ** 0.5 if E > 1 else np.ones(1)
    return p / p.sum()


def _levels(codebook):
    """The level of each 16-bit state, binary16 values."""
    s = np.arange(65536, dtype=np.uint64)
    if codebook == "mul1":
        h = (s * 0x9E3779B1) & 0xFFFFFFFF
        beta = ((h & 255) + ((h >> 8) & 255) + ((h >> 16) & 255) + (h >> 24)).astype(np.int64)
        s1, s2 = int(beta.sum()), int((beta * beta).sum())
        return ((65536 * beta - s1) / math.sqrt(65536 * s2 - s1 * s1)).astype(np.float16)
    a, b = {"mcg": (0x9E378FED, 0), "3inst": (89226354, 64248484)}[codebook]
    w = (((s * a + b) & 0x8FFF8FFF) ^ 0x3B603B60).astype(np.uint32)
    halves = w.view(np.uint16).reshape(-1, 2).view(np.float16).astype(np.float64)
    return halves.sum(axis=1).astype(np.float16)


_contexts = {}


def _context(codebook):
    """The context a program keeps, one for each codebook it uses."""
    if codebook not in _contexts:
        import trellis_coded_weight_amd as T
        _contexts[codebook] = T.Context(0)
        _contexts[codebook].set_codebook_kind(codebook)
    return _contexts[codebook]


def _inputs(case, seed):
    c = case
    n, R, C, E, K = c["n"], c["rows"], c["cols"], c["experts"], c["K"]
    dt = TYPES[c["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(c)
    # every bit string is a container; su carries the output channels' rms, a few channels are dead
    words = torch.randint(-32768, 32768, (E, R // 16, C // 16, 16 * K), generator=g, device=DEV,
                          dtype=torch.int32)
    s["packed"] = words.to(torch.int16)
    su = torch.sign(normal(E, R) + 1e-30) * 0.02 * torch.exp(0.4 * normal(E, R))
    s["su"] = torch.where(torch.rand(E, R, generator=g, device=DEV) < 0.002, 0.0, su)
    s["sv"] = torch.sign(normal(E, C) + 1e-30)
    level_std = 1.0 if c["codebook"] == "mul1" else 1.24
    s["scale"] = (1.0 + 0.1 * torch.rand(E, generator=g, device=DEV)) / level_std
    # activations with a few large channels; gradients are small
    x = normal(n, C) * torch.where(torch.rand(C, generator=g, device=DEV) < 0.004, 12.0, 1.0)
    s["x"] = x.to(dt)
    s["dy"] = (normal(n, R) * 0.01).to(dt) if c["direction"] == "backward" else None
    if c["op"] == "grouped":
        host = np.random.Generator(np.random.PCG64(seed + 5))
        sizes = host.multinomial(n, host.permutation(_expert_share(E)))
        s["largest"] = int(sizes.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)
    if c["op"] == "adapters":
        m, r = c["adapters"], c["rank"]
        s["A"] = (normal(m, r, C) / math.sqrt(C)).to(dt)
        s["B"] = (normal(m, R, r) * 0.1).to(dt)
        s["alpha"] = 0.5 + torch.rand(m, generator=g, device=DEV)
        host = np.random.Generator(np.random.PCG64(seed + 6))
        # consecutive rows of one request share its adapter; one request in ten has none
        requests = min(n, m)
        which = np.where(host.random(requests) < 0.1, -1, host.permutation(m)[:requests])
        cuts = np.sort(host.integers(0, n + 1, requests - 1)) if n > requests else np.arange(1, n)
        ids = which[np.searchsorted(cuts, np.arange(n), side="right")]
        s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import trellis_coded_weight_amd as T
        s["context"] = _context(case["codebook"])
        s["weight"] = T.CodedWeight(s["packed"], s["K"], s["scale"], s["su"], s["sv"],
                                    had_block=s["had"])
        if case["op"] == "adapters":
            s["set"] = T.Adapters(s["A"], s["B"], s["alpha"])
    else:
        s["levels"] = torch.from_numpy(_levels(case["codebook"]).astype(np.float32)).to(DEV)
        s["hadamard"] = _hadamard(case["had"], torch.float32)
    return s


def _hadamard(n, dtype):
    i = torch.arange(n, device=DEV)
    bits = i[:, None] & i[None, :]
    parity = sum((bits >> b) & 1 for b in range(7)) & 1
    return (1 - 2 * parity).to(dtype) / math.sqrt(n)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    ctx, w = s["context"], s["weight"]
    back = s["direction"] == "backward"
    if s["op"] == "linear":
        return ctx.linear(s["dy"], w, transpose=True) if back else ctx.linear(s["x"], w)
    if s["op"] == "grouped":
        if back:
            return ctx.grouped_linear(s["dy"], w, s["offsets"], transpose=True)
        return ctx.grouped_linear(s["x"], w, s["offsets"])
    if back:
        return ctx.adapter_linear_backward(s["dy"], s["x"], w, s["set"], s["ids"])
    return ctx.adapter_linear(s["x"], w, s["set"], s["ids"])


def _plain_weight(s):
    """The dense weights [experts, rows, cols] in 32 bits."""
    R, C, E, K, hb = s["rows"], s["cols"], s["experts"], s["K"], s["had"]
    words = s["packed"].to(torch.int32) & 0xFFFF
    words = words.reshape(-1, 8 * K, 2).flip(2).reshape(-1, 16 * K)
    start = ((torch.arange(256, device=DEV) + 1) * K - 16) % (256 * K)
    i, off = start // 16, (start % 16).to(torch.int32)
    states = (((words[:, i] << 16) | words[:, (i + 1) % (16 * K)]) >> (16 - off)) & 0xFFFF
    w = s["levels"][states]
    w = w.reshape(E, R // 16, C // 16, 16, 16).transpose(2, 3).reshape(E, R, C)
    h = s["hadamard"]
    w = torch.matmul(w.reshape(-1, hb), h).reshape(E, R // hb, hb, C)
    w = torch.matmul(h, w).reshape(E, R, C)
    return w * s["scale"][:, None, None] * s["su"][:, :, None] * s["sv"][:, None, :]


def _plain_grouped(x, w, offsets, largest):
    """x's rows times their group's matrix w [experts, in, out], in 32 bits."""
    row = torch.arange(x.shape[0], device=DEV)
    expert = torch.searchsorted(offsets[1:].contiguous(), row.to(torch.int32), right=True)
    slot = row - offsets[expert]
    padded = torch.zeros(w.shape[0], largest, x.shape[1], device=DEV)
    padded[expert, slot] = x.float()
    return torch.bmm(padded, w.contiguous())[expert, slot]


def _run_plain(s):
    dt = TYPES[s["dtype"]]
    w = _plain_weight(s)
    back = s["direction"] == "backward"
    if s["op"] == "linear":
        return torch.matmul(s["dy"].float(), w[0]).to(dt) if back else \
            torch.matmul(s["x"].float(), w[0].t()).to(dt)
    if s["op"] == "grouped":
        if back:
            return _plain_grouped(s["dy"], w, s["offsets"], s["largest"]).to(dt)
        return _plain_grouped(s["x"], w.transpose(1, 2), s["offsets"], s["largest"]).to(dt)
    m, r, n = s["adapters"], s["rank"], s["n"]
    x, a = s["x"].float(), s["A"].float().reshape(m * r, -1)
    b = s["B"].float().transpose(1, 2).reshape(m * r, -1)
    gate = (s["ids"][:, None] == torch.arange(m, device=DEV)) * s["alpha"]
    gate = gate[:, :, None].expand(n, m, r).reshape(n, m * r)
    v = torch.matmul(x, a.t()) * gate
    if not back:
        return (torch.matmul(x, w[0].t()) + torch.matmul(v, b)).to(dt)
    dy = s["dy"].float()
    u = torch.matmul(dy, b.t()) * gate
    dx = torch.matmul(dy, w[0]) + torch.matmul(u, a)
    da = torch.matmul(u.t(), x).reshape(m, r, -1)
    db = torch.matmul(v.t(), dy).reshape(m, r, -1).transpose(1, 2)
    return dx.to(dt), da.to(dt), db.contiguous().to(dt)


def _exact_codes(s, e):
    """Expert e's levels [rows, cols] in 64 bits, from the stream's single bits."""
    R, C, K = s["rows"], s["cols"], s["K"]
    word = s["packed"][e].reshape(-1, 16 * K)[:, torch.arange(16 * K, device=DEV) ^ 1]
    bits = (word[:, :, None].to(torch.int32) >> torch.arange(15, -1, -1, device=DEV)) & 1
    bits = bits.reshape(-1, 256 * K).to(torch.int32)
    state = torch.zeros(bits.shape[0], 256, dtype=torch.int32, device=DEV)
    for k in range(16):        # bit k of S_t lies k before the stream's bit (t + 1) K - 1
        state += torch.roll(bits, k, 1)[:, K - 1::K] << k
    lv = torch.from_numpy(_levels(s["codebook"]).astype(np.float64)).to(DEV)
    tiles = lv[state].reshape(R // 16, C // 16, 16, 16)
    return tiles.permute(0, 2, 1, 3).reshape(R, C)


def _exact_product(s, e, x, back):
    """x W_e^T, or x W_e, in 64 bits, with the transforms on the activations' side."""
    hb = s["had"]
    h = _hadamard(hb, torch.float64)
    first, last = (s["su"], s["sv"]) if back else (s["sv"], s["su"])
    codes = _exact_codes(s, e)
    z = ((x * first[e].double()).reshape(-1, hb) @ h).reshape(x.shape)
    z = z @ (codes if back else codes.t())
    z = (z.reshape(-1, hb) @ h).reshape(z.shape)
    return z * last[e].double() * s["scale"][e].double()


def exact(case, seed):
    s = _inputs(case, seed)
    back = s["direction"] == "backward"
    x = (s["dy"] if back else s["x"]).double()
    if s["op"] == "linear":
        return _exact_product(s, 0, x, back)
    if s["op"] == "grouped":
        cut = s["offsets"].tolist()
        out = [_exact_product(s, e, x[cut[e]:cut[e + 1]], back)
               for e in range(s["experts"]) if cut[e + 1] > cut[e]]
        return torch.cat(out)
    out = _exact_product(s, 0, x, back)
    A, B, alpha = s["A"].double(), s["B"].double(), s["alpha"].double()
    da, db = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(s["adapters"]):
        at = (s["ids"] == a).nonzero()[:, 0]
        xa = s["x"][at].double()
        v = xa @ A[a].t() * alpha[a]
        if not back:
            out[at] += v @ B[a].t()
            continue
        u = x[at] @ B[a] * alpha[a]
        out[at] += u @ A[a]
        da[a], db[a] = u.t() @ xa, x[at].t() @ v
    return (out, da, db) if back else out
