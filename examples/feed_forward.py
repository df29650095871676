"""A feed-forward layer whose activations travel entropy-coded.

    h  = layer_norm(x)
    a  = GELU(h W1^T + b1)   as e4m3 bytes           (one product, bias, activation and cast in its epilogue)
    a' = decode(encode(a))                            (lossless: a' is a, bit for bit)
    y  = a' W2^T + b2 + x    from the e4m3 bytes      (one product, scales, bias and residual in its epilogue)

`serve` is that path; with a batch of one it is one generated token's.  `train`
is a bf16 training step of the same layer: forward with what the backward pass
needs, then the gradients of the input and of every parameter.  `serve_experts`
routes each row to one of several experts and runs their first products as one
grouped product.

    python examples/feed_forward.py [rows] [width] [hidden]
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import lossless_entropy_coding_amd as ec

E4M3 = torch.float8_e4m3fn
CHUNK = 16384


class Layer:
    """Parameters of the layer: bf16 weights, the second one also in e4m3 with a scale per output column."""

    def __init__(self, width, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.norm_weight = 1 + normal(width, scale=0.1)
        self.norm_bias = normal(width, scale=0.1)
        self.w1 = normal(hidden, width, scale=width ** -0.5).bfloat16()
        self.b1 = normal(hidden, scale=0.1)
        self.w2 = normal(width, hidden, scale=hidden ** -0.5).bfloat16()
        self.b2 = normal(width, scale=0.1)
        most = self.w2.float().abs().amax(1).clamp(min=1e-12)
        self.w2_scale = most / 448.0
        self.w2_e4m3 = (self.w2.float() / self.w2_scale[:, None]).clamp(-448, 448).to(E4M3)
        self.act_scale = torch.full((1,), 32.0, device=device)      # activations are multiplied by it before the cast
        self.act_unscale = 1 / self.act_scale


def activations(layer, x):
    """The e4m3 bytes that the layer's first half makes of x [rows, width] (bf16)."""
    h, _, _ = ec.layer_norm(x, layer.norm_weight, layer.norm_bias)
    return ec.linear(h, layer.w1, layer.b1, act="gelu", out_scale=layer.act_scale, out_dtype=torch.uint8)


def codebook(layer, x):
    """A fixed codebook from calibration rows, made once."""
    counts = ec.byte_histogram(activations(layer, x).reshape(-1))[0].cpu().tolist()
    return ec.Codebook.huffman(counts)


def serve(layer, cb, x):
    """(y, coded bytes, status): x's rows through the layer, the activations as a stream in between."""
    a = activations(layer, x)
    out, out_len, status = ec.encode(cb, a.reshape(-1), CHUNK)
    back, status2 = ec.decode(cb, out[: int(out_len.item())], a.numel())
    y = ec.linear(back.reshape(a.shape), layer.w2_e4m3, layer.b2, residual=x, x_scale=layer.act_unscale,
                  w_scale=layer.w2_scale)
    return y, int(out_len.item()), status | status2


def train(layer, x, dy):
    """(y, gradients): one bf16 forward and backward pass; dy is the gradient of y."""
    h, mean, rstd = ec.layer_norm(x, layer.norm_weight, layer.norm_bias)
    a, z = ec.linear(h, layer.w1, layer.b1, act="gelu", save_preact=True)
    y = ec.linear(a, layer.w2, layer.b2, residual=x)
    # through the second product and the GELU before it at once, then the first product, then the norm; the
    # residual's gradient is added where the norm's is stored
    dz, dw2, db2 = ec.linear_backward(dy, a, layer.w2, preact=z, act="gelu")
    dh, dw1, db1 = ec.linear_backward(dz, h, layer.w1)
    dx, dweight, dbias = ec.layer_norm_backward(dh, x, mean, rstd, layer.norm_weight, residual_grad=dy)
    return y, dict(x=dx, w1=dw1, b1=db1, w2=dw2, b2=db2, norm_weight=dweight, norm_bias=dbias)


def serve_experts(x, router, w1, b1):
    """Each row through the expert that the router rates highest: SiLU(x w1[e]^T + b1[e]), in x's order."""
    choice = ec.linear(x, router, out_dtype=torch.float32).argmax(1)
    order = torch.argsort(choice, stable=True)
    offsets = torch.zeros(w1.shape[0] + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(torch.bincount(choice, minlength=w1.shape[0]), 0)
    y = ec.grouped_linear(x[order], w1, offsets, b1, act="silu")
    return torch.empty_like(y).index_copy_(0, order, y), choice


def main(rows=512, width=2048, hidden=8192):
    layer = Layer(width, hidden)
    x = torch.randn(rows, width, device="cuda").bfloat16()
    cb = codebook(layer, torch.randn(256, width, device="cuda").bfloat16())
    y, coded, status = serve(layer, cb, x)
    print("serve: %d rows, activations %d bytes coded to %d (%.1f%% saved), status %d"
          % (rows, rows * hidden, coded, 100 - 100.0 * coded / (rows * hidden), int(status)))
    y, grads = train(layer, x, torch.randn_like(x) * 0.01)
    print("train: " + ", ".join("%s %s" % (k, list(v.shape)) for k, v in grads.items()))
    experts = 8
    w1 = (torch.randn(experts, hidden // 4, width, device="cuda") * width ** -0.5).bfloat16()
    router = (torch.randn(experts, width, device="cuda") * width ** -0.5).bfloat16()
    y, choice = serve_experts(x, router, w1, None)
    print("experts: rows %s" % torch.bincount(choice, minlength=experts).tolist())


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
