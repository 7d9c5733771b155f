"""The experts' operators as a program uses them.

serve():  an MXFP4 expert layer, one call per batch: weights are packed once, a batch is routed, packed while
          it is dispatched, multiplied (gate and up with SwiGLU, then down) and reduced by its Top-K weights.
serve_int8():  a layer with its residual: norm, router, int8 dispatch, int8 products, the weighted sum; the batch's
          calls are captured into a CUDA graph and replayed.
train():  one training step's data movement: bf16 dispatch to the experts, a linear expert (torch), the weighted
          reduction, and the backward pass of both: the rows' and the weights' gradients, then x's.
train_router():  forward and backward of the norm and of the router with its balance loss.

Run: python examples/expert_layer.py   (needs the built library and a GPU)
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_moe_layout_02_gb300 import moe  # noqa: E402


def routing(tokens, experts, topk, dev, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    logits = torch.randn((tokens, experts), generator=g, device=dev)
    top = logits.topk(topk, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()


def serve(tokens=256, experts=16, topk=2, hidden=512, inner=256, dev="cuda"):
    """Relative distance of the layer's result from the same layer on the packed weights' values in torch."""
    torch.manual_seed(0)
    gate_up = (torch.randn((experts, 2 * inner, hidden), device=dev) / hidden ** 0.5).to(torch.bfloat16)
    down = (torch.randn((experts, hidden, inner), device=dev) / inner ** 0.5).to(torch.bfloat16)
    # once: [gate rows, up rows] become alternating groups of 16 in the packed operand
    w1 = moe.Fp4Rows(2 * inner, hidden, dev, groups=experts, gated=True).pack(gate_up)
    w2 = moe.Fp4Rows(hidden, inner, dev, groups=experts).pack(down)
    shape = moe.make_shape(1, experts, tokens, topk, hidden)
    layer = moe.Buffers(shape, dev, arena_rows=0, side_arrays=False, bits=False)

    # per batch
    x = torch.randn((tokens, hidden), device=dev).to(torch.bfloat16)
    idx, weights = routing(tokens, experts, topk, dev)
    out = torch.empty_like(x)
    layer.expert_ffn_fp4(x, idx, weights, w1.q.view(experts, 2 * inner, -1), w1.sf, w2.q.view(experts, hidden, -1), w2.sf,
                         out)
    torch.cuda.synchronize()
    assert int(layer.err[0]) == moe.MOE_OK

    values = lambda op, like: op.unpack(torch.empty_like(like)).float()
    w1v, w2v = values(w1, gate_up), values(w2, down)
    xv = values(moe.Fp4Rows(tokens, hidden, dev).pack(x), x)
    want = torch.zeros((tokens, hidden), device=dev)
    for k in range(topk):
        gu = torch.bmm(w1v[idx[:, k].long()], xv[:, :, None])[:, :, 0]
        h = (torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]).to(torch.bfloat16)
        hv = values(moe.Fp4Rows(tokens, inner, dev).pack(h), h)
        want += weights[:, k:k + 1] * torch.bmm(w2v[idx[:, k].long()], hv[:, :, None])[:, :, 0]
    return float((out.float() - want).norm() / want.norm())


def train(ranks=4, experts=16, tokens=128, topk=2, hidden=256, dev="cuda"):
    """Relative distances of the gradients of the weights and of x from autograd's on the same layer."""
    torch.manual_seed(1)
    shape = moe.make_shape(ranks, experts, tokens, topk, hidden)
    buf = moe.Buffers(shape, dev, side_arrays=False)
    mats = (torch.randn((experts, hidden, hidden), device=dev) / hidden ** 0.5).to(torch.bfloat16)
    x = torch.randn((tokens, hidden), device=dev).to(torch.bfloat16)
    idx, weights = routing(tokens, experts, topk, dev, seed=1)

    # forward: rows to the experts (contiguous per expert), the experts, the weighted sum
    buf.layout(idx)
    buf.notify()
    buf.notify_expert(idx)
    buf.dispatch_expert(x, idx, weights)
    rows = int(buf.expert_part_base[-1])
    received = buf.expert_arena[:rows, :2 * hidden].contiguous().view(torch.bfloat16)
    counts = buf.num_tokens_per_expert.sum(0).tolist()
    y = torch.cat([r @ mats[e].T for e, r in enumerate(received.split(counts))])
    out = torch.empty_like(x)
    buf.combine_expert(out, idx, weights, y=y, y_row_stride=2 * hidden)

    # backward of loss = sum(out * seed): dy and dw, through the experts, then dx by the combine without weights
    seed = torch.randn((tokens, hidden), device=dev).to(torch.bfloat16)
    dy, dw = torch.empty_like(y), torch.empty_like(weights)
    moe.moe_combine_expert_grad(shape, seed, y, 2 * hidden, buf.expert_part_base, rows, buf.slot_row, idx, weights, dy,
                                2 * hidden, dw, buf.err)
    dreceived = torch.cat([r @ mats[e] for e, r in enumerate(dy.split(counts))])
    dx = torch.empty_like(x)
    moe.moe_combine_expert(shape, dreceived, 2 * hidden, buf.expert_part_base, rows, buf.slot_row, idx, None, dx, buf.err)
    torch.cuda.synchronize()
    assert int(buf.err[0]) == moe.MOE_OK

    xr, wr = x.float().requires_grad_(), weights.clone().requires_grad_()
    ref = sum(wr[:, k:k + 1] * torch.bmm(mats[idx[:, k].long()].float(), xr[:, :, None])[:, :, 0] for k in range(topk))
    (ref * seed.float()).sum().backward()
    far = lambda a, b: float((a.float() - b).norm() / b.norm())
    return far(dw, wr.grad), far(dx, xr.grad)


def serve_int8(tokens=256, experts=16, topk=2, hidden=512, inner=256, dev="cuda"):
    """Relative distance of the layer's result from the same layer on the packed values in torch."""
    torch.manual_seed(2)
    gate_up = (torch.randn((experts * 2 * inner, hidden), device=dev) / hidden ** 0.5).to(torch.bfloat16)
    down = (torch.randn((experts * hidden, inner), device=dev) / inner ** 0.5).to(torch.bfloat16)
    router = torch.randn((experts, hidden), device=dev) / hidden ** 0.5
    scale = (1 + torch.randn(hidden, device=dev) / 8).to(torch.bfloat16)
    w1 = moe.Int8Rows(2 * inner, hidden, dev, groups=experts, gated=True).pack(gate_up)
    w2 = moe.Int8Rows(hidden, inner, dev, groups=experts).pack(down)
    shape = moe.make_shape(1, experts, tokens, topk, hidden, expert_alignment=128, quant=1)
    layer, gate = moe.Buffers(shape, dev, side_arrays=False), moe.Gate(shape, dev)
    rows = moe.moe_max_expert_rows(shape)
    x, residual = [torch.randn((tokens, hidden), device=dev).to(torch.bfloat16) for _ in range(2)]
    total, y, out = [torch.empty_like(x) for _ in range(3)]
    logits = torch.empty((tokens, experts), device=dev)
    mid, back = [torch.zeros((rows, w), dtype=torch.bfloat16, device=dev) for w in (inner, hidden)]
    packed = moe.Int8Rows(rows, inner, dev)

    def batch():
        moe.moe_rms_norm(x, scale, 1e-6, y=y, residual=residual, sum_out=total)
        torch.mm(y.float(), router.T, out=logits)
        idx, weights = gate.forward(logits)
        layer.layout(idx)
        layer.notify()
        layer.notify_expert(idx)
        layer.expert_plan()
        layer.dispatch_expert(y, idx, weights)
        layer.expert_product_int8(w1, mid)
        packed.pack(mid, E=experts, plan=layer.plan)
        moe.moe_expert_product_int8(experts, hidden, inner, 0, w2.q, w2.scale, packed.q, packed.scale, rows, layer.plan, back,
                                    layer.err)
        layer.combine_expert(out, idx, weights, y=back, y_row_stride=2 * hidden)

    batch()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch()
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert int(layer.err[0]) == moe.MOE_OK

    def values(v, n):
        op = moe.Int8Rows(n, v.shape[1], dev).pack(v)
        return op.q.float() * op.scale[:, None]

    w1v, w2v = values(gate_up, experts * 2 * inner).view(experts, 2 * inner, -1), values(down, experts * hidden).view(experts, hidden, -1)
    h = x.float() + residual.float()
    yv = values((h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * scale.float()).to(torch.bfloat16), tokens)
    top = logits.topk(topk, dim=1)
    weights = torch.softmax(top.values, 1)  # of the chosen ones: normalized
    want = torch.zeros((tokens, hidden), device=dev)
    for k in range(topk):
        e = top.indices[:, k]
        gu = torch.bmm(w1v[e], yv[:, :, None])[:, :, 0]
        inner_rows = values((torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]).to(torch.bfloat16), tokens)
        want += weights[:, k:k + 1] * torch.bmm(w2v[e], inner_rows[:, :, None])[:, :, 0]
    return float((out.float() - want).norm() / want.norm())


def train_router(tokens=256, experts=24, topk=3, hidden=512, dev="cuda"):
    """Relative distances of the gradients of the logits, of the summed rows and of the norm's weight from autograd's."""
    torch.manual_seed(3)
    shape = moe.make_shape(1, experts, tokens, topk, hidden)
    gate = moe.Gate(shape, dev, balance=0.01)
    router = (torch.randn((experts, hidden), device=dev) / hidden ** 0.5).to(torch.bfloat16)
    scale = (1 + torch.randn(hidden, device=dev) / 8).to(torch.bfloat16)
    x, residual, dsum = [torch.randn((tokens, hidden), device=dev).to(torch.bfloat16) for _ in range(3)]
    total, y, dh = [torch.empty_like(x) for _ in range(3)]
    dscale = torch.empty(hidden, device=dev)

    moe.moe_rms_norm(x, scale, 1e-6, y=y, residual=residual, sum_out=total)
    logits = y.float() @ router.float().T
    _, weights = gate.forward(logits)
    dw, dloss = torch.randn((tokens, topk), device=dev), torch.ones(1, device=dev)
    dlogits = gate.backward(logits, dw, dloss)
    dy = (dlogits @ router.float()).to(torch.bfloat16)
    moe.moe_rms_norm_grad(dy, total, scale, 1e-6, dh, dweight=dscale, dsum=dsum, scratch=moe.rms_norm_grad_scratch(tokens, hidden, dev))
    torch.cuda.synchronize()

    z = logits.clone().requires_grad_()
    p = torch.softmax(z, 1)
    top = p.topk(topk, dim=1)
    used = torch.zeros(experts, device=dev).scatter_add_(0, top.indices.reshape(-1), torch.ones(tokens * topk, device=dev))
    loss = 0.01 * experts * ((used / (topk * tokens)) * p.mean(0)).sum()
    ((top.values / top.values.sum(1, keepdim=True) * dw).sum() + loss).backward()
    h, s = total.float().requires_grad_(), scale.float().requires_grad_()
    ((h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s) * dy.float()).sum().backward()
    far = lambda a, b: float((a.float() - b).norm() / b.norm())
    return far(dlogits, z.grad), far(dh, h.grad + dsum.float()), far(dscale, s.grad)


if __name__ == "__main__":
    print("expert layer against torch on the same packed values: %.2e" % serve())
    print("int8 layer against torch on the same packed values: %.2e" % serve_int8())
    print("gradients of the logits, the summed rows and the norm's weight against autograd: %.2e %.2e %.2e" % train_router())
    print("gradients of the weights and of x against autograd: %.2e %.2e" % train())
