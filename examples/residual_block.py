"""The operators around the layer, used together: a residual stack of two blocks,

    r -> norm -> [mixture-of-experts layer] -> norm, gate, residual -> norm -> [dense gated block] -> norm, gate, residual

first as a forward pass, then training the dense block with the norms around it, then serving it one token at a
time with 4-bit weights.

    python examples/residual_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_ffn_gemv_amd as moe  # noqa: E402
import synthetic as S  # noqa: E402

DEV, DT = "cuda", torch.bfloat16


def moe_layer(shape, tokens):
    """-> a function x -> y, one mixture-of-experts layer with every expert resident."""
    cfg = moe.make_cfg(shape.dim, shape.inter, shape.n_routed, shape.topk, max_tokens=tokens)
    ctx = moe.moe_create(cfg)
    arena = moe.pack_experts(cfg, S.make_experts(shape, 0).to(DEV))
    moe.moe_set_slots(ctx, arena, shape.n_routed)
    for e in range(shape.n_routed):
        moe.moe_slot_bind(ctx, e, e)
    wr, bias = (t.to(DEV) for t in S.make_router(shape, 0, 0.05, (-0.1, 0.1)))
    weights = moe.make_weights(wr, bias)

    def call(x):
        y = torch.empty_like(x)
        moe.moe_forward(ctx, weights, x, x.shape[0], y)
        return y

    call.keep = (arena, wr, bias, ctx)
    return call


def normal(g, *shape, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale + mean).to(DT)


def quantise(w, group=64):
    """[rows, cols] -> codes, scales, zero points: the nearest of 16 values between each group's ends."""
    v = w.float().view(w.shape[0], -1, group)
    lo, hi = v.amin(2, keepdim=True).clamp(max=0), v.amax(2, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).to(DT).float()
    zero = (-lo / scale).round().clamp(0, 15)
    q = (v / scale + zero).round().clamp(0, 15).to(torch.uint8).flatten(1)
    return moe.make_w4((q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scale[..., 0].to(DT).contiguous(),
                       zero[..., 0].to(torch.uint8).contiguous(), group=group)


def main(steps=30, tokens=96, verbose=True):
    g = torch.Generator(device=DEV).manual_seed(0)
    shape = S.TINY
    dim, inter = shape.dim, 512
    w_gate, w_up = (normal(g, inter, dim, scale=dim ** -0.5) for _ in range(2))
    w_down = normal(g, dim, inter, scale=inter ** -0.5)
    w_post, w_pre = (normal(g, dim, scale=0.05, mean=1.0) for _ in range(2))
    gate = normal(g, dim, scale=0.02, mean=0.5)
    r = normal(g, tokens, dim)

    # forward: the first norm, the experts, what lies between two blocks, the dense block, the end
    first = moe.make_norm(dim, DT, w_pre=w_pre)
    between = moe.make_norm(dim, DT, w_post=w_post, w_pre=w_pre)
    last = moe.make_norm(dim, DT, w_post=w_post)
    block = moe.make_ffn(w_gate, w_up, w_down, act="silu", limit=10.0)
    forward, saved_bytes, backward = moe.moe_ffn_workspace(block, tokens)
    work = torch.empty(max(forward, backward, moe.moe_norm_workspace(last, tokens)), dtype=torch.uint8, device=DEV)
    x, y = torch.empty_like(r), torch.empty_like(r)
    moe.moe_norm_forward(first, r, None, None, x)
    y = moe_layer(shape, tokens)(x)
    moe.moe_norm_forward(between, r, y, r, x, gate=gate)   # r in place
    moe.moe_ffn_forward(block, x, y, work)
    out = torch.empty_like(r)
    moe.moe_norm_forward(last, r, y, out, None, gate=gate)

    # training: the dense block, the norm after it and its gate learn to reach a target from the r and x above
    target = out.float() + 0.5 * torch.randn(out.shape, generator=g, device=DEV)
    params = [w_gate, w_up, w_down, w_post, gate]
    master = [p.float() for p in params]
    grads = [torch.empty_like(p) for p in params]
    saved = torch.empty(saved_bytes, dtype=torch.uint8, device=DEV)
    stats = torch.empty((tokens, 2), device=DEV)
    dy = torch.empty_like(y)
    losses = []
    for _ in range(steps):
        moe.moe_ffn_forward(block, x, y, work, saved=saved)
        moe.moe_norm_forward(last, r, y, out, None, gate=gate, stats=stats)
        error = out.float() - target
        losses.append(error.square().mean().item())
        moe.moe_norm_backward(last, r, y, stats, error.to(DT), None, work, gate=gate, dy=dy, dgate=grads[4], dw_post=grads[3])
        moe.moe_ffn_backward(block, x, dy, saved, work, dw_gate=grads[0], dw_up=grads[1], dw_down=grads[2])
        for p, m, d in zip(params, master, grads):
            m.sub_(d.float(), alpha=2e-3)
            p.copy_(m)
    if verbose:
        print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")

    # serving: one token at a time through the same block with 4-bit weights
    q_gate, q_up, q_down = (quantise(w) for w in (w_gate, w_up, w_down))
    moe.moe_ffn_forward(block, x, y, work)
    h, y4 = torch.empty((1, inter), dtype=DT, device=DEV), torch.empty_like(y)
    for t in range(tokens):
        moe.moe_w4_gated(q_gate, q_up, x[t:t + 1], h, act="silu", limit=10.0)
        moe.moe_w4_matmul(q_down, h, y4[t:t + 1])
    off = ((y4.float() - y.float()).norm() / y.float().norm()).item()
    if verbose:
        print(f"serving with 4-bit weights: {off:.3f} of the block's output away from 16 bits")
    return losses, off


if __name__ == "__main__":
    main()
