"""One block of a mixture of experts on the library's operators, in training and in serving.

    python examples/expert_block.py

Training.  The residual stream h and the last block's output y meet in ``hq_block_norm`` (post norm, gate,
residual, pre norm; it also takes the amax of the rotated result, so the quantizer needs one pass).  The
normalised rows, sorted by expert, go through ``hq_grouped_gemm_nvfp4``.  Backward, the rows' gradients are the
same product with the transposed weights, the weights' gradients are ``hq_grouped_wgrad_nvfp4``, and
``hq_block_norm_bwd`` carries the gradients to h, y and the norms' parameters.  Every product's operands are
rotated and quantized along the axis that it sums over; the weights stay in bf16 beside that.

Serving.  The same norm, then a projection that all requests share with a low-rank adapter per request
(``hq_lora_gemm_nvfp4``), then the experts.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hadamard_rotation_gb300 as hq  # noqa: E402

GROUP = 16  # of the rotation


def weights_of(w):
    """Weights [E, N, K] for a product that sums over K: codes, scales in the tile layout, per-tensor scales."""
    parts = [hq.hq_rotate_quant_nvfp4_swizzled(e, GROUP, hq.hq_rot_amax(e, GROUP)) for e in w]
    return (torch.stack([p[0] for p in parts]), torch.stack([p[1].view(-1) for p in parts]),
            torch.cat([p[2] for p in parts]))


def tokens_last(x, where, T):
    """x [M, C] transposed to [C, T], each row at its place ``where`` among zeros, quantized along the tokens."""
    t = torch.zeros(x.shape[1], T, dtype=x.dtype, device=x.device)
    t[:, where] = x.t()
    q, s, sg = hq.hq_rotate_quant_nvfp4_swizzled(t, GROUP, hq.hq_rot_amax(t, GROUP))
    return q, s.view(-1), sg


class Norms(torch.autograd.Function):
    """h' = h + gate * norm(y) w_post, n = norm(h') w_pre, and the amax of the rotated n."""

    @staticmethod
    def forward(ctx, h, y, w_post, gate, w_pre):
        h_out, n, r_post, r_pre, amax = hq.hq_block_norm(h, y, w_post, gate, w_pre, amax_group=GROUP)
        ctx.save_for_backward(h_out, y, w_post, gate, w_pre, r_post, r_pre)
        ctx.mark_non_differentiable(amax)
        return h_out, n, amax

    @staticmethod
    def backward(ctx, dh_out, dn, _):
        h_out, y, w_post, gate, w_pre, r_post, r_pre = ctx.saved_tensors
        dh, dy, dw_post, dgate, dw_pre = hq.hq_block_norm_bwd(dh_out.contiguous(), dn.contiguous(), h_out, y, w_post,
                                                              gate, w_pre, r_post, r_pre)
        return dh, dy, *(g.to(w.dtype) for g, w in ((dw_post, w_post), (dgate, gate), (dw_pre, w_pre)))


class Experts(torch.autograd.Function):
    """Rows of x, sorted by expert, times their expert's weights [E, N, K] transposed."""

    @staticmethod
    def forward(ctx, x, amax, w, offsets, where, padded):
        xq, xs, x_sg = hq.hq_rotate_quant_nvfp4(x, GROUP, amax)
        ctx.save_for_backward(x, w, offsets, where, padded)
        return hq.hq_grouped_gemm_nvfp4(xq, xs, x_sg, *weights_of(w), offsets, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets, where, padded = ctx.saved_tensors
        dy = dy.contiguous()
        gq, gs, g_sg, _ = hq.hq_quantize_nvfp4(dy, GROUP)
        dx = hq.hq_grouped_gemm_nvfp4(gq, gs, g_sg, *weights_of(w.transpose(1, 2).contiguous()), offsets,
                                      out_dtype=x.dtype)
        T = int(padded[-1])
        dw = hq.hq_grouped_wgrad_nvfp4(*tokens_last(dy, where, T), *tokens_last(x, where, T), padded, out_dtype=w.dtype)
        return dx, None, dw, None, None, None


def routing(expert, E):
    """Rows' experts [M] -> (order by expert, offsets, rows' places among tokens padded to 128, their offsets)."""
    order = torch.argsort(expert, stable=True)
    sizes = torch.bincount(expert, minlength=E)

    def starts(n):
        return torch.cat([n.new_zeros(1), n.cumsum(0)])

    first, padded = starts(sizes), starts((sizes + 127) // 128 * 128)
    where = torch.arange(len(expert), device=expert.device) + (padded[:-1] - first[:-1])[expert[order]]
    return order, first.int(), where, padded.int()


def parameters(D, E, seed=0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

    return {"w_post": 1 + draw(D, scale=0.1), "gate": draw(D, scale=0.5), "w_pre": 1 + draw(D, scale=0.1),
            "w": draw(E, D, D, scale=D ** -0.5)}


def block(h, y, p, route):
    """(h', the experts' output), both [M, D]; the rows are sorted by expert."""
    h, n, amax = Norms.apply(h, y, p["w_post"], p["gate"], p["w_pre"])
    return h, Experts.apply(n, amax, p["w"], *route)


def train(steps=30, M=777, D=256, E=6, lr=0.1, device="cuda"):
    """Fits the block to one of other parameters; returns the losses."""
    g = torch.Generator(device).manual_seed(1)
    h, y = (torch.randn(M, D, generator=g, device=device).to(torch.bfloat16) for _ in range(2))
    _, *route = routing(torch.randint(0, E - 1, (M,), generator=g, device=device), E)  # (the last expert is idle)
    with torch.no_grad():
        target = block(h, y, parameters(D, E, seed=2, device=device), route)[1].float()
    p = {k: v.float().requires_grad_() for k, v in parameters(D, E, device=device).items()}
    losses = []
    for _ in range(steps):
        out = block(h, y, {k: v.to(torch.bfloat16) for k, v in p.items()}, route)[1]
        loss = (out.float() - target).square().mean()
        grads = torch.autograd.grad(loss, list(p.values()))
        with torch.no_grad():
            for w, dw in zip(p.values(), grads):
                w -= lr * D * dw
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve(h, y, p, shared, adapters, row_adapter, expert):
    """One step of M requests, a token each: norms, the shared projection with the requests' adapters, experts.

    ``shared`` [D, D] weights, ``adapters`` (A [n, R, D], B [n, D, R], scaling [n]); returns (h', output)."""
    h, n, _, _, amax = hq.hq_block_norm(h, y, p["w_post"], p["gate"], p["w_pre"], amax_group=GROUP)
    xq, xs, x_sg = hq.hq_rotate_quant_nvfp4(n, GROUP, amax)
    wq, ws, w_sg = weights_of(shared[None])
    z = hq.hq_lora_gemm_nvfp4(xq, xs, x_sg, wq[0], ws[0], w_sg, n, *adapters, row_adapter)
    order, offsets, _, _ = routing(expert, len(p["w"]))
    zq, zs, z_sg, _ = hq.hq_quantize_nvfp4(z[order], GROUP)
    out = torch.empty_like(z)
    out[order] = hq.hq_grouped_gemm_nvfp4(zq, zs, z_sg, *weights_of(p["w"]), offsets)
    return h, out


def main():
    losses = train()
    print("training: loss", " ".join(f"{v:.4f}" for v in losses[::5] + losses[-1:]))
    D, E, M, R = 256, 6, 33, 16
    g = torch.Generator("cuda").manual_seed(3)

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    adapters = (draw(4, R, D, scale=D ** -0.5), draw(4, D, R, scale=0.5), torch.ones(4, device="cuda"))
    row_adapter = (torch.arange(M, device="cuda", dtype=torch.int32) // 5) % 5 - 1  # some rows without one
    h, out = serve(draw(M, D), draw(M, D), parameters(D, E), draw(D, D, scale=D ** -0.5), adapters, row_adapter,
                   torch.randint(0, E, (M,), generator=g, device="cuda"))
    print("serving:", tuple(h.shape), tuple(out.shape), "rms", f"{float(out.float().square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
