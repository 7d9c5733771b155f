"""Cases of the operators around the experts: the router's gate, the norm before it, 8-bit products, each with what follows.

Each operator has a plain form here (elementary torch operations, binary32) and the call that a
user of the library makes; `own` says which of the two run() takes. prepare() makes what a program
holds before the call.

gate:    logits to Top-K ids, weights, per-expert counts and the balance loss; with "train" its gradient too.
norm:    root-mean-square norm of x + residual; bf16, or int8 with a scale per row (and the values back);
         with "train" bf16 and the gradient.
product: rows and weights in int8, a scale per row and per output channel, over the experts' rows or dense.
mlp:     norm to int8, gate and up, pack to int8, down: the dense (shared) expert's chain.

int8 rows: q = rint(v / scale), scale = max|v| / 127 of the row. Rows of the dispatch's int8 slots hold
`width` codes and the scale at byte ceil(width / 32) * 32, slots a multiple of 512 bytes apart. Gated
weights hold 16 gate rows and the 16 up rows that belong to them by turns.
"""

import math

import torch

own = False

TILE = 128  # experts' rows start at multiples of this
EPS = 1e-6
INF = float("inf")


# ---------------------------------------------------------------------------
# The cases


def listed():
    return [
        # The token being decoded: routing of one row of the benchmark's 256 experts.
        dict(name="gate_token", op="gate", tokens=1, experts=256, topk=8, bf16=False, train=False, normalize=True,
             masked=0.0, banned=0.0),
        # A padded batch of odd sizes, 16-bit logits (many ties), experts that a token may not use, a training step.
        dict(name="gate_ragged_train", op="gate", tokens=4999, experts=250, topk=6, bf16=True, train=True,
             normalize=False, masked=0.1, banned=0.3),
        # Forward and backward over a batch of eight ranks of the benchmark's size.
        dict(name="gate_262144x256_train", op="gate", tokens=262144, experts=256, topk=8, bf16=False, train=True,
             normalize=True, masked=0.0, banned=0.0),
        # The token being decoded, before attention or the experts.
        dict(name="norm_token", op="norm", rows=1, width=7168, residual=True, quant=False, train=False),
        # A training step on odd sizes.
        dict(name="norm_4099x2056_train", op="norm", rows=4099, width=2056, residual=True, quant=False, train=True),
        # The benchmark's batch, int8 rows for the products.
        dict(name="norm_32768x7168_int8", op="norm", rows=32768, width=7168, residual=True, quant=True, train=False),
        # A training step of half the benchmark's batch.
        dict(name="norm_16384x7168_train", op="norm", rows=16384, width=7168, residual=True, quant=False, train=True),
        # The shared expert's gate and up for the token being decoded: the weights' bytes.
        dict(name="product_token_gated", op="product", experts=0, tokens=1, topk=1, width=7168, out=4096, gated=True,
             slots=False, skew=False),
        # A decoding batch over the benchmark's experts, rows as the int8 dispatch leaves them.
        dict(name="product_decode_gated", op="product", experts=256, tokens=64, topk=8, width=7168, out=4096, gated=True,
             slots=True, skew=False),
        # Hot experts and a long tail (Zipf), the down projection.
        dict(name="product_skew_down", op="product", experts=256, tokens=1001, topk=8, width=2048, out=7168, gated=False,
             slots=False, skew=True),
        # The benchmark's batch through gate and up: the largest product.
        dict(name="product_batch_gated", op="product", experts=256, tokens=32768, topk=8, width=7168, out=4096, gated=True,
             slots=True, skew=False),
        # The shared expert's whole chain at a few hundred rows.
        dict(name="mlp_500x7168x2048", op="mlp", rows=500, width=7168, inner=2048),
    ]


def _log(rng, lo, hi):
    """A count spread over its logarithm; odd beyond a few tiles, so that it fills none."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if n > 48 else n


def draw(rng):
    op = rng.choice(["gate", "norm", "product", "product", "mlp"])
    if op == "gate":
        experts = _log(rng, 4, 1024)
        return dict(op=op, tokens=_log(rng, 1, min(262144, 262144 * 256 // experts)), experts=experts,
                    topk=rng.randint(1, min(16, experts)), bf16=rng.random() < 0.5, train=rng.random() < 0.7,
                    normalize=rng.random() < 0.6, masked=rng.choice([0.0, 0.1, 0.5]), banned=rng.choice([0.0, 0.0, 0.3]))
    if op == "norm":
        train = rng.random() < 0.5
        quant = not train and rng.random() < 0.6
        width = (16 if quant else 8) * _log(rng, 8, 448)
        return dict(op=op, rows=_log(rng, 1, min(65536, 16384 * 7168 // width)), width=width, residual=rng.random() < 0.7,
                    quant=quant, train=train)
    if op == "mlp":
        return dict(op=op, rows=_log(rng, 1, 8192), width=32 * _log(rng, 4, 224), inner=32 * _log(rng, 2, 128))
    experts = rng.choice([0, 0, 1, 2, 3, 8, 16, 60, 128, 256])
    skew = experts > 1 and rng.random() < 0.4
    gated = rng.random() < 0.5
    return dict(op=op, experts=experts, tokens=_log(rng, 1, 2048 if skew else 16384), topk=rng.randint(1, min(8, max(1, experts))),
                width=32 * _log(rng, 2, 224), out=32 * _log(rng, 2, 128), gated=gated, slots=rng.random() < 0.5, skew=skew)


# ---------------------------------------------------------------------------
# What a program holds before the call


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _generator(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=_dev())


def _codes(shape, g):
    """Random int8 codes as rows of normal values have them: the largest at 127, sigma a fourth of that."""
    out = torch.empty(shape, dtype=torch.int8, device=_dev())
    flat = out.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        part = flat[a:a + step]
        part.copy_(_normal(part.shape, g).mul_(127 / 4).round_().clamp_(-127, 127))
    return out


def _scales(shape, mid, g):
    return torch.rand(shape, generator=g, device=_dev()).add_(0.5).mul_(mid)


def _routing(case, g):
    """topk ids int32 [S, K], distinct experts by Gumbel-top-K."""
    S, E, K = case["tokens"], case["experts"], case["topk"]
    keys = -torch.log(-torch.log(torch.rand((S, E), generator=g, device=_dev()).clamp_(1e-12, 1 - 1e-7)))
    if case["skew"]:
        place = torch.randperm(E, generator=g, device=_dev())
        keys = keys - 1.2 * torch.log(place.float() + 1)
    return keys.topk(K, dim=1).indices.to(torch.int32).contiguous()


def _slot_bytes(width):
    """(bytes of a slot, byte of its scale) of the int8 dispatch."""
    at = -(-width // 32) * 32
    return -(-(at + 44) // 512) * 512, at


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "gate":
        S, E, K = case["tokens"], case["experts"], case["topk"]
        z = _normal((S, E), g).mul_(1.5).add_(_normal((E,), g).mul_(0.5))  # some experts are liked more
        if case["banned"]:
            z.masked_fill_(torch.rand((S, E), generator=g, device=_dev()) < case["banned"], -INF)
            z[torch.rand((S,), generator=g, device=_dev()) < 0.002] = -INF  # tokens that no expert may take
        s.update(logits=z.to(torch.bfloat16) if case["bf16"] else z, dw=_normal((S, K), g),
                 dloss=torch.ones((1,), device=_dev()), mask=None)
        if case["masked"]:
            s["mask"] = (torch.rand((S,), generator=g, device=_dev()) >= case["masked"]).to(torch.uint8)
        return s
    if case["op"] in ("norm", "mlp"):
        R, W = case["rows"], case["width"]
        s.update(x=_normal((R, W), g).to(torch.bfloat16), r=None, g=_normal((W,), g).mul_(0.1).add_(1).to(torch.bfloat16))
        if case.get("residual", True):
            s["r"] = _normal((R, W), g).mul_(4).to(torch.bfloat16)
        if case.get("train"):
            s.update(dy=_normal((R, W), g).to(torch.bfloat16), dsum=_normal((R, W), g).to(torch.bfloat16))
        if case["op"] == "mlp":
            inner = case["inner"]
            s.update(w1=_codes((2 * inner, W), g), w1s=_scales((2 * inner,), 4 / 127 / math.sqrt(W), g),
                     w2=_codes((W, inner), g), w2s=_scales((W,), 4 / 127 / math.sqrt(inner), g))
        return s
    S, E, K, W, N = case["tokens"], case["experts"], case["topk"], case["width"], case["out"]
    if E:
        flat = _routing(case, g).reshape(-1).long()
        counts = torch.bincount(flat, minlength=E)
        padded = (counts + TILE - 1) // TILE * TILE
        first = torch.cumsum(padded, 0) - padded
        slots = S * K
        rows = -(-(slots + min(E, slots) * (TILE - 1)) // TILE) * TILE  # rows that hold every routing
        s.update(ntpe=counts.to(torch.int32)[None].contiguous(), first=first, counts=counts)
    else:
        rows = S
        s.update(first=torch.zeros((1,), dtype=torch.int64, device=_dev()),
                 counts=torch.full((1,), S, dtype=torch.int64, device=_dev()))
    xs = _scales((rows,), 4 / 127, g)
    if case["slots"]:
        stride, at = _slot_bytes(W)
        arena = torch.zeros((rows, stride), dtype=torch.int8, device=_dev())
        arena[:, :W] = _codes((rows, W), g)
        arena[:, at:at + 4] = xs.view(torch.int8).view(rows, 4)
        s.update(arena=arena)
    else:
        s.update(xq=_codes((rows, W), g), xs=xs)
    G = max(E, 1)
    s.update(rows=rows, wq=_codes((G, N, W), g), ws=_scales((G, N), 4 / 127 / math.sqrt(W), g),
             y=torch.zeros((rows, N // 2 if case["gated"] else N), dtype=torch.bfloat16, device=_dev()))
    return s


# ---------------------------------------------------------------------------
# The plain forms


def _plain_gate(s):
    case = s["case"]
    S, E, K = case["tokens"], case["experts"], case["topk"]
    z = s["logits"].float()
    top, idx = torch.sort(z, dim=1, descending=True, stable=True)  # equal logits in the order of their ids
    top, idx = top[:, :K], idx[:, :K]
    routed = top[:, 0] > -INF
    if s["mask"] is not None:
        routed = routed & (s["mask"] != 0)
    live = routed[:, None] & (top > -INF)
    e = torch.exp(z - torch.where(routed, z.amax(1), 0)[:, None])
    p = torch.where(routed[:, None], e / e.sum(1, keepdim=True), 0)
    pk = torch.where(live, p.gather(1, idx), 0)
    norm = torch.where(routed, pk.sum(1), 1)[:, None] if case["normalize"] else torch.ones((), device=z.device)
    w = pk / norm
    ids = torch.where(live, idx, -1)
    counts = (torch.bincount(ids.reshape(-1) + 1, minlength=E + 1)[1:]).to(torch.int32)
    n = routed.sum()
    share = counts / (n.clamp_min(1) * K).float()
    prob = (p.double().sum(0) / n.clamp_min(1)).float()
    loss = 0.01 * E * (share * prob).sum()
    out = dict(idx=ids.to(torch.int32), weights=w, count=torch.cat([counts, n.to(torch.int32)[None]]), prob=prob,
               loss=loss.reshape(1))
    if case["train"]:
        dw = torch.where(live, s["dw"], 0)
        a = (dw - (dw * w).sum(1, keepdim=True) if case["normalize"] else dw) / norm
        dp = (s["dloss"] * (0.01 * E) * share / n.clamp_min(1)).expand(S, E).clone()
        dp.scatter_add_(1, idx, torch.where(live, a, 0))
        dz = p * (dp - (p * dp).sum(1, keepdim=True))
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


def _int8(v):
    """(codes, scales) of rows, binary32."""
    scale = v.abs().amax(1, keepdim=True) / 127
    return torch.where(scale > 0, torch.round(v / scale).clamp(-127, 127), 0), scale


def _normed(s):
    h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["g"].float()


def _plain_norm(s):
    case = s["case"]
    h, y = _normed(s)
    out = dict(sum=h.to(torch.bfloat16)) if s["r"] is not None else {}
    if case["quant"]:
        q, scale = _int8(y)
        out.update(values=(q * scale).to(torch.bfloat16), scale=scale[:, 0])
        return out
    out["y"] = y.to(torch.bfloat16)
    if case["train"]:
        h = h.to(torch.bfloat16).float()  # the sum as it is kept
        rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        xhat = h * rstd
        dy = s["dy"].float()
        gdy = dy * s["g"].float()
        dh = rstd * (gdy - xhat * (gdy * xhat).mean(1, keepdim=True)) + s["dsum"].float()
        out.update(dh=dh.to(torch.bfloat16), dg=(dy * xhat).double().sum(0).float())
    return out


def _gate(v):
    """[.., 2I] with 16 gate rows and 16 up rows by turns -> silu(gate) * up [.., I]."""
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 2, 16)
    return (v[..., 0, :] / (1 + torch.exp(-v[..., 0, :])) * v[..., 1, :]).reshape(*v.shape[:-3], v.shape[-3] * 16)


def _rows(s):
    """Codes and scales of the case's rows."""
    if "arena" not in s:
        return s["xq"], s["xs"]
    W = s["case"]["width"]
    at = _slot_bytes(W)[1]
    return s["arena"][:, :W], s["arena"][:, at:at + 4].contiguous().view(torch.float32)[:, 0]


def _plain_product(s):
    case = s["case"]
    q, scale = _rows(s)
    first, counts = s["first"], s["counts"]
    most = int(counts.max())
    at = torch.arange(most, device=q.device)
    mine = at[None, :] < counts[:, None]
    at = torch.where(mine, first[:, None] + at[None, :], 0)
    v = torch.bmm(q[at].float(), s["wq"].float().transpose(1, 2))
    v = v * s["ws"][:, None, :] * scale[at][:, :, None]
    if case["gated"]:
        v = _gate(v)
    y = torch.zeros_like(s["y"])
    y[at[mine]] = v[mine].to(y.dtype)
    return y


def _plain_mlp(s):
    h, y = _normed(s)
    q, scale = _int8(y)
    v = _gate(q @ s["w1"].float().T * s["w1s"] * scale).to(torch.bfloat16)  # inner rows are bf16
    q, scale = _int8(v.float())
    return dict(sum=h.to(torch.bfloat16), y=(q @ s["w2"].float().T * s["w2s"] * scale).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# The library's calls


def _own_gate(s):
    from combine_moe_layout_02_gb300 import moe

    case = s["case"]
    if "op" not in s:  # the program's buffers
        shape = moe.make_shape(1, case["experts"], case["tokens"], case["topk"], 64)
        s["op"] = moe.Gate(shape, s["logits"].device, normalize=case["normalize"], balance=0.01)
    op = s["op"]
    op.forward(s["logits"], mask=s["mask"])
    out = dict(idx=op.topk_idx, weights=op.topk_weights, count=op.expert_count, prob=op.expert_prob, loss=op.loss)
    if case["train"]:
        out["dlogits"] = op.backward(s["logits"], s["dw"], s["dloss"], mask=s["mask"])
    return out


def _own_norm(s):
    from combine_moe_layout_02_gb300 import moe

    case = s["case"]
    x, r = s["x"], s["r"]
    if "y" not in s:
        s["y"] = torch.empty_like(x)
        s["sum"] = torch.empty_like(x) if r is not None else None
        if case["quant"]:
            s["rows"] = moe.Int8Rows(case["rows"], case["width"], x.device)
        if case["train"]:
            s["dh"] = torch.empty_like(x)
            s["dg"] = torch.empty((case["width"],), dtype=torch.float32, device=x.device)
            s["scratch"] = moe.rms_norm_grad_scratch(case["rows"], case["width"], x.device)
    out = dict(sum=s["sum"]) if r is not None else {}
    if case["quant"]:
        op = s["rows"]
        moe.moe_rms_norm(x, s["g"], EPS, residual=r, sum_out=s["sum"], q=op.q, q_scale=op.scale)
        out.update(values=op.unpack(s["y"]), scale=op.scale)
        return out
    moe.moe_rms_norm(x, s["g"], EPS, y=s["y"], residual=r, sum_out=s["sum"])
    out["y"] = s["y"]
    if case["train"]:
        h = x if r is None else s["sum"]
        moe.moe_rms_norm_grad(s["dy"], h, s["g"], EPS, s["dh"], dweight=s["dg"], dsum=s["dsum"], scratch=s["scratch"])
        out.update(dh=s["dh"], dg=s["dg"])
    return out


def _own_product(s):
    from combine_moe_layout_02_gb300 import moe

    case = s["case"]
    E, N, W = case["experts"], case["out"], case["width"]
    plan = None
    if "err" not in s:
        s["err"] = torch.zeros((4,), dtype=torch.int32, device=s["y"].device)
        if E:
            s["shape"] = moe.make_shape(1, E, case["tokens"], case["topk"], 64, expert_alignment=TILE)
            s["plan"] = moe.expert_plan_buffer(s["shape"], s["y"].device)
    if E:
        plan = s["plan"]
        moe.moe_expert_plan(s["shape"], s["ntpe"], plan)
    if case["slots"]:
        stride, at = _slot_bytes(W)
        moe.moe_expert_product_int8(max(E, 1), N, W, case["gated"], s["wq"], s["ws"], s["arena"],
                                    s["arena"].data_ptr() + at, s["rows"], plan, s["y"], s["err"], x_row_stride=stride,
                                    xs_stride=stride)
    else:
        moe.moe_expert_product_int8(max(E, 1), N, W, case["gated"], s["wq"], s["ws"], s["xq"], s["xs"], s["rows"], plan,
                                    s["y"], s["err"])
    return s["y"]


def _own_mlp(s):
    from combine_moe_layout_02_gb300 import moe

    case = s["case"]
    R, W, inner = case["rows"], case["width"], case["inner"]
    if "sum" not in s:
        dev = s["x"].device
        s.update(sum=torch.empty_like(s["x"]), y=torch.empty_like(s["x"]), a=moe.Int8Rows(R, W, dev),
                 h=torch.empty((R, inner), dtype=torch.bfloat16, device=dev), b=moe.Int8Rows(R, inner, dev),
                 err=torch.zeros((4,), dtype=torch.int32, device=dev))
    a, b = s["a"], s["b"]
    moe.moe_rms_norm(s["x"], s["g"], EPS, residual=s["r"], sum_out=s["sum"], q=a.q, q_scale=a.scale)
    moe.moe_expert_product_int8(1, 2 * inner, W, True, s["w1"], s["w1s"], a.q, a.scale, R, None, s["h"], s["err"])
    b.pack(s["h"])
    moe.moe_expert_product_int8(1, W, inner, False, s["w2"], s["w2s"], b.q, b.scale, R, None, s["y"], s["err"])
    return dict(sum=s["sum"], y=s["y"])


_PLAIN = dict(gate=_plain_gate, norm=_plain_norm, product=_plain_product, mlp=_plain_mlp)
_OWN = dict(gate=_own_gate, norm=_own_norm, product=_own_product, mlp=_own_mlp)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    if case["op"] == "gate":
        S, E, K = case["tokens"], case["experts"], case["topk"]
        z = (2 if case["bf16"] else 4) * S * E
        back = z + 4 * S * K if case["train"] else 0  # the logits' gradient, dw
        return dict(bytes=float(z + back + 8 * S * K + 8 * E), flops=float((16 if case["train"] else 8) * S * E))
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        each = 2 + (4 if case["residual"] else 0) + 2 + (6 if case["train"] else 0)  # rows in and out, 2 bytes each
        return dict(bytes=float(each * n), flops=float((14 if case["train"] else 6) * n))
    if case["op"] == "mlp":
        R, W, inner = case["rows"], case["width"], case["inner"]
        return dict(bytes=float(3 * inner * W + 8 * R * W), flops=6.0 * R * inner * W)
    E, K, W, N = case["experts"], case["topk"], case["width"], case["out"]
    rows = case["tokens"] * K
    hit = E * (1 - (1 - K / E) ** case["tokens"]) if E else 1  # experts that some row goes to, were it uniform
    return dict(bytes=float(hit * N * (W + 4) + rows * (W + 4) + 2 * rows * (N // 2 if case["gated"] else N)),
                flops=2.0 * rows * N * W)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits


def _exact_gate(s):
    case = s["case"]
    S, E, K = case["tokens"], case["experts"], case["topk"]
    z = s["logits"].double().clone().requires_grad_(case["train"])
    left = s["logits"].double().clone()
    if s["mask"] is not None:
        left[s["mask"] == 0] = -INF
    ids = []
    for _ in range(K):  # the largest that is left, of equal ones the first
        most = left.amax(1, keepdim=True)
        first = (left == most).int().argmax(1)
        ids.append(torch.where(most[:, 0] > -INF, first, -1))
        left.scatter_(1, first[:, None], -INF)
    idx = torch.stack(ids, 1)
    routed, live = idx[:, 0] >= 0, idx >= 0
    n = int(routed.sum())
    full = torch.where(routed[:, None], z, torch.zeros((), dtype=torch.float64, device=z.device))
    p = torch.softmax(full, 1) * routed[:, None]
    w = p.gather(1, idx.clamp_min(0)) * live
    if case["normalize"]:
        w = w / torch.where(routed, w.sum(1), torch.ones((), dtype=torch.float64, device=z.device))[:, None]
    counts = torch.stack([(idx == e).sum() for e in range(E)])
    prob = p.sum(0) / max(n, 1)
    loss = 0.01 * E * (counts.double() / (max(n, 1) * K) * prob).sum()
    out = dict(idx=idx.to(torch.int32), weights=w.detach(), prob=prob.detach(), loss=loss.detach().reshape(1),
               count=torch.cat([counts, torch.tensor([n], device=counts.device)]).to(torch.int32))
    if case["train"]:
        (grad,) = torch.autograd.grad((w * torch.where(live, s["dw"].double(), 0)).sum() + loss * s["dloss"].double()[0], z)
        out["dlogits"] = grad
    return out


def _exact_norm(s):
    case = s["case"]
    out = {}
    h = s["x"].double()
    if s["r"] is not None:
        h = h + s["r"].double()
        out["sum"] = h
    g = s["g"].double()
    y = h * g * (h.square().sum(1, keepdim=True) / case["width"] + EPS).rsqrt()
    if case["quant"]:
        out["scale"] = y.abs().amax(1) / 127
        out["values"] = torch.round(y / out["scale"][:, None]) * out["scale"][:, None]
        return out
    out["y"] = y
    if case["train"]:
        h = h.to(torch.bfloat16).double().requires_grad_()
        g = g.clone().requires_grad_()
        y = h * g * (h.square().sum(1, keepdim=True) / case["width"] + EPS).rsqrt()
        dh, dg = torch.autograd.grad((y * s["dy"].double()).sum(), (h, g))
        out.update(dh=dh + s["dsum"].double(), dg=dg)
    return out


def _exact_linear(codes, scale, wq, ws, gated):
    """The sums are whole numbers: 1024 products of codes are below 2^24, which binary32 holds, and these add up in 64 bits."""
    v = torch.zeros((codes.shape[0], wq.shape[0]), dtype=torch.float64, device=wq.device)
    for a in range(0, wq.shape[1], 1024):
        v += codes[:, a:a + 1024].float() @ wq[:, a:a + 1024].float().T
    v = v * ws.double() * scale.double()[:, None]
    if not gated:
        return v
    i = torch.arange(v.shape[1] // 2, device=v.device)
    at = i // 16 * 32 + i % 16
    return v[:, at] * torch.sigmoid(v[:, at]) * v[:, at + 16]


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e13 or (case["op"] in ("gate", "norm") and w["bytes"] > 6e9):
        return None  # too long in 64 bits
    s = prepare(case, seed)
    if case["op"] == "gate":
        return _exact_gate(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "mlp":
        h = s["x"].double() + s["r"].double()
        y = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * s["g"].double()
        scale = y.abs().amax(1) / 127
        v = _exact_linear(torch.round(y / scale[:, None]), scale, s["w1"], s["w1s"], True)
        v = v.to(torch.bfloat16).double()  # inner rows are bf16 before they are packed
        scale = v.abs().amax(1) / 127
        return dict(sum=h, y=_exact_linear(torch.round(v / scale[:, None]), scale, s["w2"], s["w2s"], False))
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
    q, scale = _rows(s)
    for e in torch.nonzero(s["counts"]).flatten().tolist():
        a, b = int(s["first"][e]), int(s["first"][e] + s["counts"][e])
        y[a:b] = _exact_linear(q[a:b], scale[a:b], s["wq"][e], s["ws"][e], case["gated"])
    return y
