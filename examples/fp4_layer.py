"""A pre-norm residual layer on microscaled 4-bit products: trained for some
steps, then run one token at a time.

    h(x) = x + W . layer_norm(x) + b

    python examples/fp4_layer.py [--rows 2048] [--width 1024] [--steps 30] [--fmt nv|mx]

Training keeps W, gamma, beta and b in fp32, packs W anew for every step in
both directions, and learns another such layer from its outputs.  The forward
pass quantizes the norm's output inside the linear call; the backward pass
quantizes the gradient in both directions for its two products.  A single token
goes through the norm straight to codes and through a product of packed
operands: two kernels.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bit_quantized_tensor_gb300 as qg  # noqa: E402


class Layer:
    def __init__(self, width, fmt, seed, dev):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.fmt = fmt
        self.W = torch.randn(width, width, generator=g, device=dev) / width ** 0.5
        self.b = torch.zeros(width, device=dev)
        self.gamma = torch.ones(width, device=dev)
        self.beta = torch.zeros(width, device=dev)
        self.pack()

    def scale(self, X):
        return qg.fp4_tensor_scale(X) if self.fmt == "nv" else None

    def pack(self):
        """W's codes along its rows (forward) and along its columns (backward)."""
        self.ws = self.scale(self.W)
        self.Wq, self.Ws, self.Wtq, self.Wts = qg.fp4_quantize_both(self.W, self.fmt, scale=self.ws)

    def forward(self, x):
        y, mean, rstd = qg.layer_norm(x, self.gamma, self.beta)
        ys = self.scale(y)
        out = qg.fp4_linear(y, self.Wq, self.Ws, self.fmt, x_scale=ys, w_scale=self.ws, bias=self.b.to(x.dtype))
        return x + out, (x, y, ys, mean, rstd)

    def backward(self, dh, saved):
        x, y, ys, mean, rstd = saved
        dy, dW, db = qg.fp4_linear_backward(dh, y, self.Wtq, self.Wts, self.fmt, dy_scale=self.scale(dh),
                                            x_scale=ys, w_scale=self.ws)
        dx, dgamma, dbeta = qg.layer_norm_backward(dy, x, self.gamma, mean, rstd)
        return dh + dx, dW, db, dgamma, dbeta

    def token(self, x):
        q, s, _, _ = qg.layer_norm_fp4(x, self.gamma, self.beta, fmt=self.fmt)
        return x + qg.fp4_gemm(q, s, self.Wq, self.Ws, x.shape[1], self.fmt, b_scale=self.ws, bias=self.b.to(x.dtype),
                               dtype=x.dtype)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--fmt", choices=("nv", "mx"), default="nv")
    a = ap.parse_args(argv)
    if not torch.cuda.is_available():
        sys.exit("fp4_layer needs a CUDA device")
    dev = torch.device("cuda:0")
    teacher, layer = Layer(a.width, a.fmt, 1, dev), Layer(a.width, a.fmt, 2, dev)
    g = torch.Generator(device=dev).manual_seed(3)
    rate, losses = 0.5, []  # the norm's output has unit variance, so 1 would be a Newton step
    for _ in range(a.steps):
        x = torch.randn(a.rows, a.width, generator=g, device=dev).to(torch.bfloat16)
        want = x + torch.nn.functional.layer_norm(x.float(), (a.width,)) @ teacher.W.t()
        h, saved = layer.forward(x)
        diff = h.float() - want
        losses.append(float(diff.square().mean()))
        dh = (diff / a.rows).to(torch.bfloat16)  # of half the squared difference, mean over rows
        _, dW, db, dgamma, dbeta = layer.backward(dh, saved)
        layer.W -= rate * dW.float()
        layer.b -= rate * db
        layer.gamma -= 0.1 * dgamma / a.width
        layer.beta -= 0.1 * dbeta / a.width
        layer.pack()
    x = torch.randn(4, a.width, generator=g, device=dev).to(torch.bfloat16)
    batch, _ = layer.forward(x)
    singles = torch.cat([layer.token(x[i:i + 1]) for i in range(4)])
    apart = float((batch.float() - singles.float()).norm() / batch.float().norm())
    if qg.device_status() != qg.QG_OK:
        sys.exit(f"device status {qg.device_status()}")
    print(f"{a.fmt}: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; "
          f"tokens one at a time against the batch: {apart:.4f} apart")
    return losses, apart


if __name__ == "__main__":
    main()
