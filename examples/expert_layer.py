"""The experts' operators as a program uses them.

serve():  an MXFP4 expert layer, one call per batch: weights are packed once, a batch is routed, packed while
          it is dispatched, multiplied (gate and up with SwiGLU, then down) and reduced by its Top-K weights.
train():  one training step's data movement: bf16 dispatch to the experts, a linear expert (torch), the weighted
          reduction, and the backward pass of both: the rows' and the weights' gradients, then x's.

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


if __name__ == "__main__":
    print("expert layer against torch on the same packed values: %.2e" % serve())
    print("gradients of the weights and of x against autograd: %.2e %.2e" % train())
