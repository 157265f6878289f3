"""A small expert layer on coded weights: quantize, run a prompt and single tokens, train adapters.

The layer is a projection with low-rank adapters beside it (one per request), a router, and one
matrix per expert; every large matrix is held as trellis codes.

    python examples/coded_layer.py [--rows 1024] [--experts 8] [--tokens 512] [--bits 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import trellis_coded_weight_amd as T  # noqa: E402


def signs(n, generator):
    return torch.randint(0, 2, (n,), generator=generator, device="cuda").float() * 2 - 1


def quantize(context, w, bits, generator):
    """A dense matrix [rows, cols] -> (container, scale, su, sv), the rows' rms folded into su."""
    su, sv = signs(w.shape[0], generator), signs(w.shape[1], generator)
    w_norm, su_folded, _ = context.channel_normalize(w, su)
    out = context.quantize_matrix(w_norm, bits, su, sv)
    return out["packed"], out["scale"], su_folded, sv


class ExpertLayer:
    def __init__(self, context, dim, experts, bits, requests, rank, generator):
        self.context, self.experts = context, experts

        def dense():
            w = torch.randn(dim, dim, generator=generator, device="cuda") * dim ** -0.5
            return w.bfloat16()

        self.dense_proj = dense()
        self.proj = T.CodedWeight(*self._coded([self.dense_proj], bits, generator))
        self.dense_experts = [dense() for _ in range(experts)]
        self.mlp = T.CodedWeight(*self._coded(self.dense_experts, bits, generator, grouped=True))
        self.router = torch.randn(experts, dim, generator=generator, device="cuda").bfloat16()
        self.A = (torch.randn(requests, rank, dim, generator=generator, device="cuda") *
                  dim ** -0.5).bfloat16().requires_grad_()
        self.B = torch.zeros(requests, dim, rank, device="cuda",
                             dtype=torch.bfloat16).requires_grad_()
        self.alpha = torch.ones(requests, device="cuda")

    def _coded(self, matrices, bits, generator, grouped=False):
        parts = [quantize(self.context, w, bits, generator) for w in matrices]
        if not grouped:
            packed, scale, su, sv = parts[0]
            return packed, bits, scale, su, sv
        packed, scale, su, sv = zip(*parts)
        return (torch.stack(packed), bits, torch.tensor(scale, device="cuda"), torch.stack(su),
                torch.stack(sv))

    def __call__(self, x, ids):
        """x [tokens, dim], ids int32 [tokens]: the request of each token, or -1."""
        h = T.coded_adapter_linear(self.context, x, self.proj, self.A, self.B, self.alpha, ids)
        expert = (h.float() @ self.router.float().t()).argmax(dim=1)
        order = torch.argsort(expert, stable=True)
        sizes = torch.bincount(expert, minlength=self.experts)
        offsets = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()
        y = T.coded_grouped_linear(self.context, h[order], self.mlp, offsets)
        return torch.zeros_like(y).index_copy(0, order, y), expert

    def dense(self, x, expert):
        """The same with the matrices before quantization, for comparison."""
        h = x.float() @ self.dense_proj.float().t()
        out = torch.empty_like(h)
        for e in range(self.experts):
            out[expert == e] = h[expert == e] @ self.dense_experts[e].float().t()
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--bits", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    generator = torch.Generator(device="cuda")
    generator.manual_seed(1)
    with T.Context(0) as context:
        layer = ExpertLayer(context, a.rows, a.experts, a.bits, 4, 8, generator)
        x = torch.randn(a.tokens, a.rows, generator=generator, device="cuda").bfloat16()
        ids = (torch.arange(a.tokens, device="cuda") * 5 // a.tokens - 1).int()

        with torch.no_grad():
            y, expert = layer(x, ids)
            ref = layer.dense(x, expert)
            off = float((y.float() - ref).norm() / ref.norm())
            print("prompt of %d tokens, K = %d: %.3f of the dense layer's norm off" %
                  (a.tokens, a.bits, off))
            one = torch.cat([layer(x[t:t + 1], ids[t:t + 1])[0] for t in range(4)])
            same = float((one.float() - y[:4].float()).norm() / y[:4].float().norm())
            print("four single tokens against the prompt: %.2g" % same)

        # adapters learn to bring the layer's first projection to a target
        target = (x.float() @ torch.randn(a.rows, a.rows, generator=generator, device="cuda") *
                  a.rows ** -0.5).bfloat16()
        optimizer = torch.optim.Adam([layer.A, layer.B], lr=1e-3)
        losses = []
        for _ in range(a.steps):
            h = T.coded_adapter_linear(context, x, layer.proj, layer.A, layer.B, layer.alpha, ids)
            loss = ((h - target).float() ** 2)[ids >= 0].mean()
            optimizer.zero_grad()
            loss.backward()
            optimizer.step()
            losses.append(float(loss.detach()))
        print("adapters: loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))
        torch.cuda.synchronize()
    return off, same, losses


if __name__ == "__main__":
    main()
