"""A stack of feed-forward blocks on the 8-bit integer path, as a serving program
would run it, and the training step of the boundary between two blocks.

Serving, per layer (weights quantised once per channel):

    h, hs = norm(x) * w_pre                 block_norm, h in 8 bits with its scales
    u     = relu(h @ W_up^T)                gemm_i8
    y     = u @ W_down^T                    linear_i8 (quantises u itself)
    x     = alpha x + gate * norm(y) * w_post   block_norm, together with the next
                                            layer's norm: x and h in one pass

A token that is not finite keeps its infinities and NaN in the residual stream
only: in 8 bits its row has the scale NaN, and the ReLU after the first product
takes NaN to zero.

Training runs the same boundary with h in the block's type and takes its
gradients (block_norm_backward).

    python -m tiled_dense_gemm_07_amd.int8_block [--tokens 256] [--width 4096]
        [--hidden 8192] [--layers 4]

prints the time of a pass and how far it is from the same stack in fp32.
"""

from __future__ import annotations

import argparse
import time

from . import binding


class Int8Stack:
    """Layers of random weights: `width` in and out, `hidden` between."""

    def __init__(self, width: int, hidden: int, layers: int, seed: int = 0, device="cuda",
                 alpha: float = 1.0):
        import torch

        g = torch.Generator(device=device)
        g.manual_seed(seed)
        bf16 = torch.bfloat16
        self.width, self.alpha = width, alpha
        self.layers = []
        for _ in range(layers):
            w_up = torch.randn((hidden, width), generator=g, device=device) / width ** 0.5
            w_down = torch.randn((width, hidden), generator=g, device=device) / hidden ** 0.5
            layer = {"up": w_up, "down": w_down}
            layer["up_q"], layer["up_s"] = binding.quant_i8(w_up)  # a scale for each channel
            layer["down_q"], layer["down_s"] = binding.quant_i8(w_down)
            for name, add, scale in (("w_pre", 1.0, 0.1), ("w_post", 1.0, 0.1), ("gate", 0.0, 0.5)):
                v = add + scale * torch.randn((width,), generator=g, device=device)
                layer[name] = v.to(bf16)
            self.layers.append(layer)

    def serve(self, x):
        """x [T, width] bf16 through every layer; returns the residual stream."""
        f = binding.block_norm(x, w_pre=self.layers[0]["w_pre"], out="i8")
        for i, layer in enumerate(self.layers):
            u = binding.gemm_i8(f.h, f.hs, layer["up_q"], layer["up_s"], epilogue="relu")
            y = binding.linear_i8(u, layer["down_q"], layer["down_s"])
            more = i + 1 < len(self.layers)
            f = binding.block_norm(
                f.x, y=y, gate=layer["gate"], w_post=layer["w_post"], alpha=self.alpha,
                w_pre=self.layers[i + 1]["w_pre"] if more else None, out="i8" if more else None)
        return f.x

    def plain(self, x):
        """The same stack in fp32 torch operations, nothing quantised."""
        norm = lambda v: v * (v.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt()
        x = x.float()
        for layer in self.layers:
            u = (norm(x) * layer["w_pre"].float()) @ layer["up"].t()
            y = u.clamp(min=0.0) @ layer["down"].t()
            x = self.alpha * x + layer["gate"].float() * norm(y) * layer["w_post"].float()
        return x

    def boundary_step(self, x, y, dx_new, dh, layer: int = 0):
        """Training step of the boundary after `layer`: (forward, gradients)."""
        a, b = self.layers[layer], self.layers[(layer + 1) % len(self.layers)]
        f = binding.block_norm(x, y=y, gate=a["gate"], w_post=a["w_post"], w_pre=b["w_pre"],
                               alpha=self.alpha, save=True)
        g = binding.block_norm_backward(f.x, dx_new, dh, y=y, gate=a["gate"], w_post=a["w_post"],
                                        w_pre=b["w_pre"], r_post=f.r_post, r_pre=f.r_pre,
                                        alpha=self.alpha)
        return f, g


def main(argv=None) -> int:
    import torch

    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--layers", type=int, default=4)
    args = ap.parse_args(argv)
    stack = Int8Stack(args.width, args.hidden, args.layers)
    x = torch.randn((args.tokens, args.width), device="cuda").to(torch.bfloat16)

    def timed(f, n=20):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6

    out, want = stack.serve(x).float(), stack.plain(x)
    off = ((out - want).norm() / want.norm()).item()
    print("serving %d tokens, %d layers of %d x %d: %.1f us in 8 bits, %.1f us in fp32; %.2f%% apart"
          % (args.tokens, args.layers, args.width, args.hidden, timed(lambda: stack.serve(x)),
             timed(lambda: stack.plain(x)), 100.0 * off))
    y, dx, dh = (torch.randn_like(x) for _ in range(3))
    print("training step of one boundary: %.1f us"
          % timed(lambda: stack.boundary_step(x, y, dx, dh)))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
