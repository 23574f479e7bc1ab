"""A transformer block whose tokens look at a prompt's states, on the INT8 linears:

    q, k, v = x W_q, (c W_k, c W_v as one packed linear)
    q, k    = per-head norms, q rotated by its tokens' positions   (ck_qk_norm_rope)
    x       = x + attention(q, k, v) W_o                           (ck_cross_attn; residual in the linear)
    x       = x + SwiGLU MLP(x)

``python examples/cross_block.py`` runs it on synthetic data and compares it with the same block in FP32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_mlp_amd as ck  # noqa: E402


class CrossBlock:
    """weights: FP32 tensors w_q [h d, width], w_kv [2 h d, context], w_o [width, h d], w_gu [2 i, width],
    w_down [width, i] and the head norms g_q, g_k [d]."""

    def __init__(self, weights, heads, group=128):
        self.heads, self.group = heads, group
        self.norms = weights["g_q"], weights["g_k"]
        self.w = {n: ck.ck_weight_prep(w, group) for n, w in weights.items() if w.dim() == 2}

    def _linear(self, x, name, residual=None):
        return ck.ck_int8_linear(x, *self.w[name], self.group, residual=residual)

    def __call__(self, x, context, rope, context_len=None):
        """x [batch, tokens, width], context [batch, states, width of its own], both BF16; rope: (cos, sin) of the
        tokens; context_len int32 [batch]: the states of each prompt."""
        b, t, width = x.shape
        s = context.shape[1]
        flat = x.reshape(b * t, width)
        q = self._linear(flat, "w_q").view(b, t, self.heads, -1)
        kv = self._linear(context.reshape(b * s, -1), "w_kv").view(b, s, 2 * self.heads, -1)
        k, v = kv[:, :, :self.heads], kv[:, :, self.heads:]
        # one launch for both, in place in the projections' outputs
        ck.ck_qk_norm_rope(q, k, *self.norms, q_rope=rope, q_out=q, k_out=k)
        o = ck.ck_cross_attn(q, k, v, kv_len=context_len)
        flat = self._linear(o.view(b * t, -1), "w_o", residual=flat)
        mlp = ck.ck_swiglu_mlp(flat, *self.w["w_gu"], *self.w["w_down"], self.group)
        return (flat + mlp).view(b, t, width)


def reference(weights, heads, x, context, rope, context_len):
    """The block in FP32 with the unquantized weights."""
    b, t, width = x.shape
    x = x.float()

    def norm(y, g):
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * g

    q = norm((x @ weights["w_q"].T).view(b, t, heads, -1), weights["g_q"])
    k, v = (context.float() @ weights["w_kv"].T).view(b, context.shape[1], 2, heads, -1).unbind(2)
    k = norm(k, weights["g_k"])
    cos, sin = (r[:t, None] for r in rope)
    half = cos.shape[-1]
    a, c = q[..., :half], q[..., half:]
    q = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    scores = q.transpose(1, 2) @ k.permute(0, 2, 3, 1).contiguous() * q.shape[-1] ** -0.5
    states = torch.arange(k.shape[1], device=x.device)
    scores.masked_fill_(states >= context_len[:, None, None, None], float("-inf"))
    o = torch.softmax(scores, -1) @ v.transpose(1, 2).contiguous()
    x = x + o.transpose(1, 2).reshape(b, t, -1) @ weights["w_o"].T
    gate, up = (x @ weights["w_gu"].T).chunk(2, -1)
    return x + (torch.nn.functional.silu(gate) * up) @ weights["w_down"].T


def synthetic(b=2, t=1024, s=77, heads=8, d=128, context=512, inner=2048, seed=0):
    """(weights, x, context, rope, context_len) on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = heads * d

    def rand(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=g, device="cuda")

    weights = {"w_q": rand(width, width, scale=0.03), "w_kv": rand(2 * width, context, scale=0.04),
               "w_o": rand(width, width, scale=0.03), "w_gu": rand(2 * inner, width, scale=0.03),
               "w_down": rand(width, inner, scale=0.02), "g_q": 1 + 0.2 * rand(d), "g_k": 1 + 0.2 * rand(d)}
    angle = torch.arange(t, device="cuda")[:, None] * torch.pow(10000.0, -torch.arange(0, d, 2, device="cuda") / d)
    lens = torch.linspace(s // 2, s, b, device="cuda").to(torch.int32)
    return weights, rand(b, t, width).bfloat16(), rand(b, s, context).bfloat16(), (angle.cos(), angle.sin()), lens


def main():
    heads = 8
    weights, x, context, rope, lens = synthetic(heads=heads)
    block = CrossBlock(weights, heads)
    y = block(x, context, rope, lens)
    want = reference(weights, heads, x, context, rope, lens)
    print(f"relative L2 against FP32: {((y.float() - want).norm() / want.norm()).item():.4f}", flush=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(50):
        block(x, context, rope, lens)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / 50 * 1e3:.1f} us a block of {x.shape[0]} x {x.shape[1]} tokens over "
          f"{context.shape[1]} states")


if __name__ == "__main__":
    main()
