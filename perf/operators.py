"""Cases of the experts' operators: MXFP4 packing, the grouped product, the expert FFN, combine's gradient.

Each operator has a plain form here (elementary torch operations, binary32) and the call that a
user of the library makes; `own` says which of the two run() takes. prepare() makes what a program
holds before the call: rows, routing, packed weights, the tables of the forward pass.

MXFP4 operands (OCP Microscaling Formats v1.0: e2m1 elements, one ue8m0 scale per 32) are held as
the library documents them: `q` uint8 [rows, width / 2], the even element in the low nibble; `sf`
uint8 [ceil(rows / 128), ceil(width / 128), 512], where row m's scale of block 4c + j is byte
(m % 32) * 16 + (m % 128) / 32 * 4 + j of chunk c.
"""

import math

import numpy as np
import torch

own = False

TILE = 128  # experts' rows start at multiples of this
NAN = float("nan")


# ---------------------------------------------------------------------------
# The cases


def listed():
    return [
        # A few activation rows of the smallest configuration: launch latency.
        dict(name="pack_16x256", op="pack", rows=16, width=256, wide=False),
        # Rows and width that fill no tile (the width ends inside a chunk of scales), values over many binades.
        dict(name="pack_1001x2080_wide", op="pack", rows=1001, width=2080, wide=True),
        # The hidden rows of the benchmark's batch.
        dict(name="pack_32768x7168", op="pack", rows=32768, width=7168, wide=False),
        # One token being decoded: 8 experts' gate and up weights are read for one row each.
        dict(name="product_token_gated", op="product", ranks=8, experts=256, tokens=8, live=1, topk=8, width=7168,
             out=4096, gated=True, skew=False),
        # A decoding batch: most experts are hit, by two rows or so each; the weights' bytes are the time.
        dict(name="product_decode_gated", op="product", ranks=8, experts=256, tokens=64, live=64, topk=8, width=7168,
             out=4096, gated=True, skew=False),
        # Hot experts and a long tail (Zipf), the down projection: row counts from none to all tokens.
        dict(name="product_skew_down", op="product", ranks=32, experts=256, tokens=1024, live=1001, topk=8, width=2048,
             out=7168, gated=False, skew=True),
        # The benchmark's batch through gate and up: the largest product.
        dict(name="product_batch_gated", op="product", ranks=8, experts=256, tokens=32768, live=32768, topk=8,
             width=7168, out=4096, gated=True, skew=False),
        # The whole expert layer at the smallest configuration: the latency of the call chain.
        dict(name="ffn_p4_t64", op="ffn", ranks=4, experts=16, tokens=256, topk=2, width=256, inner=128, skew=False,
             masked=0.0),
        # The whole expert layer at the small-message configuration.
        dict(name="ffn_p32_t128", op="ffn", ranks=32, experts=256, tokens=4096, topk=8, width=7168, inner=2048,
             skew=False, masked=0.0),
        # Combine's gradient at the smallest configuration, one row per (token, slot).
        dict(name="grad_p4_t64", op="grad", layout="expert", ranks=4, experts=16, tokens=256, topk=2, width=256,
             weighted=True, skew=False, masked=0.0),
        # Combine's gradient over 128 ranks with hot ranks and masked slots, one row per (token, rank).
        dict(name="grad_p128_rank_skew", op="grad", layout="rank", ranks=128, experts=256, tokens=8192, topk=8,
             width=7168, weighted=True, skew=True, masked=0.1),
        # Combine's gradient of a large batch, one row per (token, slot).
        dict(name="grad_p8_expert", op="grad", layout="expert", ranks=8, experts=256, tokens=16384, topk=8, width=7168,
             weighted=True, skew=False, masked=0.0),
    ]


def _log(rng, lo, hi):
    """A count spread over its logarithm; odd beyond a few tiles, so that it fills none."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if n > 48 else n


def draw(rng):
    op = rng.choice(["pack", "product", "ffn", "grad"])
    if op == "pack":
        width = 32 * _log(rng, 2, 448)
        rows = _log(rng, 1, min(65536, 32768 * 7168 // width))
        return dict(op=op, rows=rows, width=width, wide=rng.random() < 0.5)
    ranks = rng.choice([1, 2, 4, 8, 16, 32])
    experts = ranks * rng.choice([n for n in (1, 2, 3, 4, 8, 16, 32, 64) if 8 <= n * ranks <= 256])
    topk = rng.randint(1, 8)
    if op == "product":
        skew = rng.random() < 0.4
        gated = rng.random() < 0.5
        width, out = 32 * _log(rng, 4, 224), 32 * _log(rng, 4, 128)
        per = _log(rng, 1, max(2, (2048 if skew else 16384) // ranks))
        live = rng.randint(max(1, ranks * per // 2), ranks * per)
        return dict(op=op, ranks=ranks, experts=experts, tokens=ranks * per, live=live, topk=topk, width=width, out=out,
                    gated=gated, skew=skew)
    if op == "ffn":
        per = _log(rng, 1, max(2, 4096 // ranks))
        return dict(op=op, ranks=ranks, experts=experts, tokens=ranks * per, topk=topk, width=32 * _log(rng, 4, 224),
                    inner=32 * _log(rng, 2, 64), skew=rng.random() < 0.3, masked=rng.choice([0.0, 0.1]))
    per = _log(rng, 1, max(2, 16384 // ranks))
    return dict(op=op, layout=rng.choice(["expert", "rank"]), ranks=ranks, experts=experts, tokens=ranks * per,
                topk=topk, width=8 * _log(rng, 8, 896), weighted=rng.random() < 0.8, skew=rng.random() < 0.4,
                masked=rng.choice([0.0, 0.1, 0.5]))


# ---------------------------------------------------------------------------
# What a program holds before the call


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _generator(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    return g


def _routing(case, g):
    """topk ids int32 [S, K] (distinct experts by Gumbel-top-K; -1 where masked) and softmax weights [S, K]."""
    S, E, K = case["tokens"], case["experts"], case["topk"]
    keys = -torch.log(-torch.log(torch.rand((S, E), generator=g, device=_dev()).clamp_(1e-12, 1 - 1e-7)))
    if case["skew"]:
        place = torch.randperm(E, generator=g, device=_dev())
        keys = keys - 1.2 * torch.log(place.float() + 1)
    idx = keys.topk(K, dim=1).indices.to(torch.int32)
    if case.get("masked"):
        idx[torch.rand((S, K), generator=g, device=_dev()) < case["masked"]] = -1
    if case.get("live", S) < S:
        idx[case["live"]:] = -1
    w = torch.softmax(torch.randn((S, K), generator=g, device=_dev()), 1)
    return idx.contiguous(), w.contiguous()


def _expert_rows(idx, experts, tile):
    """Rows of the expert-major layout: per slot its row (-1 where masked), each expert's first row and count, all rows."""
    flat = idx.reshape(-1).long()
    counts = torch.bincount(flat[flat >= 0], minlength=experts)
    padded = (counts + tile - 1) // tile * tile
    first = torch.cumsum(padded, 0) - padded
    order = torch.sort(torch.where(flat >= 0, flat, experts), stable=True).indices
    order = order[: int(counts.sum())]
    rank = torch.arange(order.numel(), device=idx.device) - (torch.cumsum(counts, 0) - counts)[flat[order]]
    row = torch.full_like(flat, -1)
    row[order] = first[flat[order]] + rank
    return row.reshape(idx.shape), first, counts, int(padded.sum())


def _codes(shape, g):
    """Random packed e2m1 pairs: each element drawn as a normal value would be rounded (sigma = 1/3 of the largest code)."""
    edges = [0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, math.inf]
    mass = [math.erf(b / 2 / math.sqrt(2)) - math.erf(a / 2 / math.sqrt(2)) for a, b in zip(edges, edges[1:])]
    table = np.searchsorted(np.cumsum(mass), (np.arange(128) + 0.5) / 128).clip(0, 7).astype(np.uint8)
    table = torch.from_numpy(np.concatenate([table, table + 8])).to(_dev())
    table = (table[:, None] | (table[None, :] << 4)).reshape(-1)  # by 16 random bits
    out = torch.empty(shape, dtype=torch.uint8, device=_dev())
    rows = max(1, (1 << 28) // max(1, math.prod(shape[1:])))
    for a in range(0, shape[0], rows):
        part = out[a:a + rows]
        part.copy_(table[torch.randint(0, 65536, part.shape, generator=g, device=_dev(), dtype=torch.int32)])
    return out


def _scales(shape, width, mid, g):
    """Random scale codes near `mid` in the tiled layout of [..., rows, width] operands; 0 past the width."""
    *lead, rows = shape
    sf = torch.full((*lead, -(-rows // 128), -(-width // 128), 32, 4, 4), mid, dtype=torch.uint8, device=_dev())
    sf += torch.randint(0, 3, sf.shape, generator=g, device=_dev(), dtype=torch.uint8)
    if width % 128:
        sf[..., -1, :, :, width % 128 // 32:] = 0
    return sf.reshape(*sf.shape[:-3], 512)


def _hidden(rows, width, g):
    return torch.randn((rows, width), generator=g, device=_dev()).to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "pack":
        s["x"] = _hidden(case["rows"], case["width"], g)
        if case["wide"]:
            e = torch.randint(-24, 25, (case["rows"], case["width"] // 32, 1), generator=g, device=_dev())
            s["x"] = (s["x"].float().reshape(*e.shape[:2], 32) * torch.exp2(e.float())).to(torch.bfloat16)
            s["x"] = s["x"].reshape(case["rows"], case["width"]).contiguous()
        s["y"] = torch.empty_like(s["x"])
        return s
    S, E, P, K, W = case["tokens"], case["experts"], case["ranks"], case["topk"], case["width"]
    idx, w = _routing(case, g)
    if case["op"] == "product":
        _, first, counts, _ = _expert_rows(idx, E, TILE)
        N = case["out"]
        slots = case["live"] * K
        total = -(-(slots + min(E, slots) * (TILE - 1)) // TILE) * TILE  # rows that hold every routing
        src = torch.arange(S, device=_dev()) // (S // P)
        ntpe = torch.zeros((P, E), dtype=torch.int32, device=_dev())
        live = idx >= 0
        ntpe.view(-1).index_add_(0, (src[:, None].expand(S, K)[live] * E + idx[live].long()),
                                 torch.ones(int(live.sum()), dtype=torch.int32, device=_dev()))
        s.update(ntpe=ntpe, first=first, counts=counts, rows=total, q=_codes((total, W // 2), g),
                 sf=_scales((total,), W, 125, g), wq=_codes((E, N, W // 2), g),
                 wsf=_scales((E, N), W, 126 - int(math.log2(W) / 2), g),
                 y=torch.zeros((total, N // 2 if case["gated"] else N), dtype=torch.bfloat16, device=_dev()))
        return s
    if case["op"] == "ffn":
        inner = case["inner"]
        s.update(x=_hidden(S, W, g), idx=idx, w=w, out=torch.empty((S, W), dtype=torch.bfloat16, device=_dev()),
                 w1=_codes((E, 2 * inner, W // 2), g), w1sf=_scales((E, 2 * inner), W, 126 - int(math.log2(W) / 2), g),
                 w2=_codes((E, W, inner // 2), g), w2sf=_scales((E, W), inner, 126 - int(math.log2(inner) / 2), g))
        return s
    # combine's gradient: the forward pass's rows, tables and weights, and the gradient of its result
    s.update(idx=idx, w=w if case["weighted"] else None, dout=_hidden(S, W, g))
    if case["layout"] == "expert":
        row, first, counts, total = _expert_rows(idx, E, 1)
        base = torch.cat([first.reshape(P, E // P)[:, 0], first.new_full((1,), total)])
        e = idx.long().clamp_min(0) // (E // P)
        s.update(base=base.contiguous(), slot_row=torch.where(row >= 0, row - base[e], row).to(torch.int32).contiguous())
    else:
        sent = torch.zeros((S, P + 1), dtype=torch.bool, device=_dev())
        sent.scatter_(1, torch.where(idx >= 0, idx // (E // P), P).long(), True)
        sent = sent[:, :P]
        per = sent.sum(0)
        head = torch.where(sent, torch.cumsum(sent.long(), 0) - 1, -1)
        s.update(base=torch.cat([per.new_zeros(1), torch.cumsum(per, 0)]).contiguous(), head=head.to(torch.int32).contiguous())
    rows = S * (K if case["layout"] == "expert" else min(K, P))  # rows that hold every routing
    s.update(rows=rows, y=_hidden(rows, W, g), dy=torch.zeros((rows, W), dtype=torch.bfloat16, device=_dev()),
             dw=torch.zeros((S, K), dtype=torch.float32, device=_dev()))
    return s


# ---------------------------------------------------------------------------
# The plain forms


def _grid(device):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    v = torch.cat([v, -v])
    return torch.stack([v[torch.arange(256, device=device) & 15], v[torch.arange(256, device=device) >> 4]], 1)


def _power(code):
    """2 ** (code - 127) in binary32; NaN for 255."""
    v = (code.to(torch.int32) << 23).view(torch.float32)
    v = torch.where(code == 0, 2.0 ** -127, v)
    return torch.where(code == 255, NAN, v)


def _flat_scales(sf, rows, width):
    """Tiled scales [..., tiles, chunks, 512] to [..., rows, width / 32]."""
    lead, (tiles, chunks) = sf.shape[:-3], sf.shape[-3:-1]
    n = len(lead)
    v = sf.reshape(*lead, tiles, chunks, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return v.reshape(*lead, tiles * 128, chunks * 4)[..., :rows, : width // 32]


def _values(q, sf):
    """A packed operand's values in binary32."""
    rows, width = q.shape[-2], q.shape[-1] * 2
    v = _grid(q.device)[q.int()].reshape(*q.shape[:-1], width // 32, 32)
    return (v * _power(_flat_scales(sf, rows, width))[..., None]).reshape(*q.shape[:-1], width)


def _rounded(x):
    """Rows rounded to MXFP4, as the values they then stand for, in binary32."""
    v = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    exponent = (v.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) & 255
    code = torch.where(exponent == 255, 255, (exponent - 2).clamp_min(0))
    scale = _power(code)
    back = torch.where(code == 255, NAN, _power((254 - code).clamp_min(0)))
    a = (v * back).abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp_max(6)
    return (torch.copysign(a, v) * scale).reshape(x.shape)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _by_expert(rows, first, counts):
    """Row numbers [E, most] of each expert (0 past its count) and which of them are its own."""
    most = max(1, int(counts.max()))
    at = torch.arange(most, device=rows.device)
    mine = at[None, :] < counts[:, None]
    return torch.where(mine, first[:, None] + at[None, :], 0), mine


def _gate(v):
    """[.., 2I] with 16 gate rows and 16 up rows by turns -> silu(gate) * up [.., I]."""
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 2, 16)
    return (_silu(v[..., 0, :]) * v[..., 1, :]).reshape(*v.shape[:-3], v.shape[-3] * 16)


def _product(x, w, first, counts, gated, y):
    """y's rows of each expert from rows x [rows, width] and weights w [E, out, width]."""
    at, mine = _by_expert(x, first, counts)
    v = torch.bmm(x[at], w.transpose(1, 2))
    if gated:
        v = _gate(v)
    y[at[mine]] = v[mine].to(y.dtype)
    return y


def _plain(s):
    case = s["case"]
    if case["op"] == "pack":
        return _rounded(s["x"]).to(torch.bfloat16)
    if case["op"] == "product":
        return _product(_values(s["q"], s["sf"]), _values(s["wq"], s["wsf"]), s["first"], s["counts"], case["gated"],
                        torch.zeros_like(s["y"]))
    S, K, E, P = case["tokens"], case["topk"], case["experts"], case["ranks"]
    idx = s["idx"]
    if case["op"] == "ffn":
        row, first, counts, total = _expert_rows(idx, E, 1)
        live = row >= 0
        x = torch.zeros((max(total, 1), case["width"]), device=idx.device)
        x[row[live]] = _rounded(s["x"])[:, None, :].expand(S, K, case["width"])[live]
        h = torch.zeros((max(total, 1), case["inner"]), dtype=torch.bfloat16, device=idx.device)
        h = _product(x, _values(s["w1"], s["w1sf"]), first, counts, True, h)
        y = torch.zeros((max(total, 1), case["width"]), dtype=torch.bfloat16, device=idx.device)
        y = _product(_rounded(h), _values(s["w2"], s["w2sf"]), first, counts, False, y)
        w = torch.where(live, s["w"], 0)
        return torch.bmm(w[:, None, :], y[row.clamp_min(0)].float())[:, 0].to(torch.bfloat16)
    epr = E // P
    live = idx >= 0
    rank = idx.long().clamp_min(0) // epr
    w = s["w"] if s["w"] is not None else torch.ones((S, K), device=idx.device)
    if case["layout"] == "expert":
        row = torch.where(live, s["base"][rank] + s["slot_row"], 0)
        scale = w
    else:
        row = torch.where(live, s["base"][rank] + s["head"].gather(1, rank), 0)
        same = (rank[:, :, None] == rank[:, None, :]) & live[:, None, :]
        scale = (same * w[:, None, :]).sum(-1) if s["w"] is not None else w
    token = torch.arange(S, device=idx.device)[:, None].expand(S, K)
    dy = torch.zeros_like(s["dy"])
    dy[row[live]] = (scale[live][:, None] * s["dout"].float()[token[live]]).to(dy.dtype)
    dots = torch.zeros((S, K), device=idx.device)
    dots[live] = (s["dout"].float()[token[live]] * s["y"].float()[row[live]]).sum(-1)
    return dict(dy=dy, dw=dots) if s["w"] is not None else dict(dy=dy)


# ---------------------------------------------------------------------------
# The library's calls


def _own(s):
    from combine_moe_layout_02_gb300 import moe

    case = s["case"]
    if case["op"] == "pack":
        if "op" not in s:  # the program's buffers
            s["op"] = moe.Fp4Rows(case["rows"], case["width"], s["x"].device)
        s["op"].pack(s["x"])
        return s["op"].unpack(s["y"])
    if "shape" not in s:
        s["shape"] = moe.make_shape(case["ranks"], case["experts"], case["tokens"], case["topk"], case["width"],
                                    expert_alignment=TILE if case["op"] != "grad" else 1)
    shape = s["shape"]
    if case["op"] == "product":
        if "plan" not in s:
            s["plan"] = moe.expert_plan_buffer(shape, s["y"].device)
            s["err"] = torch.zeros((4,), dtype=torch.int32, device=s["y"].device)
        moe.moe_expert_plan(shape, s["ntpe"], s["plan"])
        moe.moe_expert_product_fp4(case["experts"], case["out"], case["width"], case["gated"], s["wq"], s["wsf"],
                                   s["q"], s["sf"], s["rows"], s["plan"], s["y"], s["err"])
        return s["y"]
    if case["op"] == "ffn":
        if "buf" not in s:
            s["buf"] = moe.Buffers(shape, s["x"].device, arena_rows=0, side_arrays=False, bits=False)
        s["buf"].expert_ffn_fp4(s["x"], s["idx"], s["w"], s["w1"], s["w1sf"], s["w2"], s["w2sf"], s["out"])
        return s["out"]
    if "err" not in s:
        s["err"] = torch.zeros((4,), dtype=torch.int32, device=s["y"].device)
    dw = s["dw"] if s["w"] is not None else None
    if case["layout"] == "expert":
        moe.moe_combine_expert_grad(shape, s["dout"], s["y"], 2 * case["width"], s["base"], s["rows"], s["slot_row"],
                                    s["idx"], s["w"], s["dy"], 2 * case["width"], dw, s["err"])
    else:
        moe.moe_combine_grad(shape, s["dout"], s["y"], 2 * case["width"], s["base"], s["rows"], s["head"], s["idx"],
                             s["w"], s["dy"], 2 * case["width"], dw, s["err"])
    return dict(dy=s["dy"], dw=dw) if dw is not None else dict(dy=s["dy"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def _fp4_bytes(rows, width):
    return rows * width * 17 / 32


def work(case):
    W = case["width"]
    if case["op"] == "pack":  # rows in, the values out
        return dict(bytes=4.0 * case["rows"] * W, flops=0.0)
    S, K, E, P = case["tokens"], case["topk"], case["experts"], case["ranks"]
    live = case.get("live", S) * K * (1 - case.get("masked", 0.0))
    # experts that some row goes to, for a uniform routing (a skewed one reaches fewer)
    hit = E * (1 - (1 - K / E) ** (live / K))
    if case["op"] == "product":
        N = case["out"]
        back = N // 2 if case["gated"] else N
        return dict(bytes=hit * _fp4_bytes(N, W) + _fp4_bytes(live, W) + 2 * live * back, flops=2.0 * live * N * W)
    if case["op"] == "ffn":
        inner = case["inner"]
        return dict(bytes=hit * (_fp4_bytes(2 * inner, W) + _fp4_bytes(W, inner)) + 4.0 * S * W + 8.0 * S * K,
                    flops=6.0 * live * inner * W)
    rows = live if case["layout"] == "expert" else S * P * (1 - (1 - 1 / P) ** (live / S))
    return dict(bytes=2.0 * S * W + 4.0 * rows * W + 12.0 * S * K, flops=3.0 * rows * W)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits


def _two_to(n):
    """2 ** n for whole n, by its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_operand(q, sf, rows, width):
    """e2m1: sign, two bits of exponent (bias 1), one bit of fraction; times 2 ** (scale - 127)."""
    c = torch.stack([q % 16, q // 16], -1).reshape(rows, width).long()
    e, f = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, f / 2, (1 + f / 2) * _two_to(e - 1))
    m, k = torch.arange(rows, device=q.device)[:, None], torch.arange(width // 32, device=q.device)[None, :]
    byte = sf[m // 128, k // 4, (m % 32) * 16 + m % 128 // 32 * 4 + k % 4]
    return torch.where(c >= 8, -mag, mag) * _two_to(byte.long() - 127).repeat_interleave(32, 1)


def _exact_rounded(x):
    """The nearest e2m1 value under the block's power of two, ties to the even code, at most 6."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    v = x.double().reshape(-1, 32)
    most = v.abs().amax(1, keepdim=True)
    unit = _two_to((torch.frexp(most).exponent.long() - 3).clamp_min(-127))  # frexp's fraction is in [1/2, 1)
    a = v.abs() / unit
    low, high = torch.bucketize(a, middle), torch.bucketize(a, middle, right=True)
    code = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return (torch.sign(v) * grid[code] * unit).reshape(x.shape)


def _exact_product(x, operand, first, counts, gated, y):
    for e in torch.nonzero(counts).flatten().tolist():
        a, n = int(first[e]), int(counts[e])
        v = x(a, n) @ operand(e).T
        if gated:
            i = torch.arange(v.shape[1] // 2, device=v.device)
            at = i // 16 * 32 + i % 16
            gate, up = v[:, at], v[:, at + 16]
            v = gate / (1 + torch.exp(-gate)) * up
        y[a:a + n] = v
    return y


def exact(case, seed):
    flops = work(case)["flops"]
    if flops > 4e12 or (case["op"] in ("pack", "grad") and work(case)["bytes"] > 6e9):
        return None  # too long in 64 bits
    s = prepare(case, seed)
    W = case["width"]
    if case["op"] == "pack":
        return _exact_rounded(s["x"])
    E, S, K, P = case["experts"], case["tokens"], case["topk"], case["ranks"]
    dev = _dev()
    if case["op"] == "product":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=dev)
        return _exact_product(lambda a, n: _exact_operand(s["q"][a:a + n], s["sf"][a // 128:], n, W),
                              lambda e: _exact_operand(s["wq"][e], s["wsf"][e], case["out"], W),
                              s["first"], s["counts"], case["gated"], y)
    idx = s["idx"]
    if case["op"] == "ffn":
        inner = case["inner"]
        slots = [torch.nonzero(idx.flatten() == e).flatten() for e in range(E)]
        counts = torch.tensor([len(v) for v in slots])
        first = torch.cumsum(counts, 0) - counts
        slot = torch.cat(slots)
        rows = len(slot)
        x = _exact_rounded(s["x"])[slot // K]
        h = torch.zeros((rows, inner), dtype=torch.float64, device=dev)
        h = _exact_product(lambda a, n: x[a:a + n], lambda e: _exact_operand(s["w1"][e], s["w1sf"][e], 2 * inner, W),
                           first, counts, True, h)
        h = _exact_rounded(h.to(torch.bfloat16))  # the experts' inner rows are bf16 before they are packed
        y = torch.zeros((rows, W), dtype=torch.float64, device=dev)
        y = _exact_product(lambda a, n: h[a:a + n], lambda e: _exact_operand(s["w2"][e], s["w2sf"][e], W, inner),
                           first, counts, False, y)
        out = torch.zeros((S, W), dtype=torch.float64, device=dev)
        return out.index_add_(0, slot // K, s["w"].flatten()[slot][:, None].double() * y)
    dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device=dev)
    dw = torch.zeros((S, K), dtype=torch.float64, device=dev)
    for k in range(K):
        g = torch.nonzero(idx[:, k] >= 0).flatten()
        d = idx[g, k].long() // (E // P)
        place = s["slot_row"][g, k] if case["layout"] == "expert" else s["head"][g, d]
        row = s["base"][d] + place
        w = s["w"][g, k].double() if s["w"] is not None else torch.ones(len(g), dtype=torch.float64, device=dev)
        back = s["dout"][g].double()
        dw[g, k] = (back * s["y"][row].double()).sum(1)
        if case["layout"] == "rank" and s["w"] is not None:
            dy.index_add_(0, row, w[:, None] * back)  # a rank's weight is the sum of its slots'
        else:
            dy[row] = w[:, None] * back
    return dict(dy=dy, dw=dw) if s["w"] is not None else dict(dy=dy)
