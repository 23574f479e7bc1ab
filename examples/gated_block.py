"""An image transformer block with modulated norms, on MX FP4 linears:

    h       = norm(x) (1 + scale_a) + shift_a                          (ck_block_norm)
    q, k, v = h W_qkv;  q, k = per-head norms with positions           (ck_mx4_linear, ck_qk_norm_rope)
    x, h    = x + gate_a attention(q, k, v) W_o, its modulated norm    (ck_cross_attn, ck_mx4_linear, ck_block_norm)
    x       = x + gate_m SwiGLU MLP(h)                                 (ck_mx4_linear twice, ck_block_norm)

The six modulations of a sequence are column ranges of one packed tensor.  ``python examples/gated_block.py`` runs it on
synthetic data and compares it with the same block in FP32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_mlp_amd as ck  # noqa: E402


class GatedBlock:
    """weights: FP32 tensors w_qkv [3 h d, width], w_o [width, h d], w_gu [2 i, width], w_down [width, i] and the head
    norms g_q, g_k [d]."""

    def __init__(self, weights, heads, group=128):
        self.heads, self.group = heads, group
        self.norms = weights["g_q"], weights["g_k"]
        self.w = {n: (*ck.ck_mx4_weight_prep(w, group), w.shape[0]) for n, w in weights.items() if w.dim() == 2}

    def _linear(self, x, name, input_act=None):
        codes, scales, n = self.w[name]
        return ck.ck_mx4_linear(x, codes, scales, n=n, group=self.group, input_act=input_act)

    def __call__(self, x, modulation, rope):
        """x [batch, tokens, width] BF16; modulation [batch, 6 width] BF16: shift, scale and gate of the attention, then of
        the MLP; rope: (cos, sin) of the tokens."""
        b, t, width = x.shape
        shift_a, scale_a, gate_a, shift_m, scale_m, gate_m = modulation.view(b, 6, width).unbind(1)
        h = ck.ck_block_norm(x, norm="layer", scale=scale_a, shift=shift_a)
        qkv = self._linear(h.view(b * t, width), "w_qkv").view(b, t, 3 * self.heads, -1)
        q, k, v = qkv.split(self.heads, 2)
        ck.ck_qk_norm_rope(q, k, *self.norms, q_rope=rope, k_rope=rope, q_out=q, k_out=k)
        o = self._linear(ck.ck_cross_attn(q, k, v).view(b * t, -1), "w_o").view(b, t, width)
        x, h = ck.ck_block_norm(x, o, gate=gate_a, norm="layer", scale=scale_m, shift=shift_m, out=o)
        y = self._linear(self._linear(h.view(b * t, width), "w_gu"), "w_down", "swiglu").view(b, t, width)
        return ck.ck_block_norm(x, y, gate=gate_m, norm=None, x_out=x)


def reference(weights, heads, x, modulation, rope):
    """The block in FP32 with the unquantized weights -> (y, its two gated branches)."""
    b, t, width = x.shape
    x = x.float()
    shift_a, scale_a, gate_a, shift_m, scale_m, gate_m = (m[:, None] for m in modulation.float().view(b, 6, width).unbind(1))

    def layer(y):
        return torch.nn.functional.layer_norm(y, (width,), eps=1e-6)

    def head(y, g):
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * g
        cos, sin = (r[:t, None] for r in rope)
        a, c = y.chunk(2, -1)
        return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)

    q, k, v = ((layer(x) * (1 + scale_a) + shift_a) @ weights["w_qkv"].T).view(b, t, 3, heads, -1).unbind(2)
    q, k = head(q, weights["g_q"]), head(k, weights["g_k"])
    s = q.transpose(1, 2) @ k.permute(0, 2, 3, 1).contiguous() * q.shape[-1] ** -0.5
    o = (torch.softmax(s, -1) @ v.transpose(1, 2).contiguous()).transpose(1, 2).reshape(b, t, -1)
    first = gate_a * (o @ weights["w_o"].T)
    x = x + first
    gate, up = ((layer(x) * (1 + scale_m) + shift_m) @ weights["w_gu"].T).chunk(2, -1)
    second = gate_m * ((torch.nn.functional.silu(gate) * up) @ weights["w_down"].T)
    return x + second, first, second


def synthetic(b=2, t=1024, heads=8, d=128, inner=2048, seed=0):
    """(weights, x, modulation, rope) on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = heads * d

    def rand(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=g, device="cuda")

    weights = {"w_qkv": rand(3 * width, width, scale=0.03), "w_o": rand(width, width, scale=0.03),
               "w_gu": rand(2 * inner, width, scale=0.03), "w_down": rand(width, inner, scale=0.02),
               "g_q": 1 + 0.2 * rand(d), "g_k": 1 + 0.2 * rand(d)}
    angle = torch.arange(t, device="cuda")[:, None] * torch.pow(10000.0, -torch.arange(0, d, 2, device="cuda") / d)
    return weights, rand(b, t, width).bfloat16(), rand(b, 6 * width, scale=0.3).bfloat16(), (angle.cos(), angle.sin())


def main():
    heads = 8
    weights, x, modulation, rope = synthetic(heads=heads)
    block = GatedBlock(weights, heads)
    y = block(x, modulation, rope)
    want, *_ = reference(weights, heads, x, modulation, rope)
    print(f"relative L2 against FP32: {((y.float() - want).norm() / want.norm()).item():.4f}", flush=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(50):
        block(x, modulation, rope)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 50 * 1e3:.1f} us a block of {x.shape[0]} x {x.shape[1]} tokens")


if __name__ == "__main__":
    main()
