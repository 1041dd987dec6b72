"""Workloads of an expert block in 8 bits: rows and weights quantised in
blocks of 128, the experts' products of them, and the norms around the block.

  quantize   rows [R, W] -> e4m3 values and, for each 128 elements of a row, a
             scale that is a power of two, the smallest with which no value
             passes 448 (one for a block of zeros); the last block of a row
             may be shorter.  Or weights [E, N, K], one scale for each 128 x
             128 elements of an expert's matrix.
  dispatch   the tokens' rows laid out by expert and quantised (dropped slots:
             zero rows).
  matmul     per expert: activation(x w^T + bias) + residual of quantised x and
             w, in 16 bits or quantised again; rows past the last expert's are
             zero.
  norm       h = rms(x) * weight, or the way out of a block and into the next
             in one: y = residual_scale * x + gate * (rms(block) *
             block_weight), h = rms(y) * weight of y as it is held; rms(v) =
             v / sqrt(mean(v^2) + eps).  A gate has one row for all, or one
             for each sequence.
  norm_grad  its gradients, given those of h and (through the residual path) y.

run() computes them with elementary torch operations in 32 bits, rounded
once at the end, or through the package when `own` is set.  exact() computes
them in 64 bits from their definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


def listed():
    return [
        # A prompt's activations before a dense product: odd counts.
        dict(name="quantize prompt odd", op="quantize", rows=5003, width=1037, dtype="f16"),
        # A layer's weights when a trained model is loaded, or after a step.
        dict(name="quantize weights", op="quantize_weights", experts=16, outer=4096, inner=2048, dtype="bf16",
             transposed=False),
        # One decoding step of 64 sequences.
        dict(name="dispatch decode", op="dispatch", tokens=64, slots=8, experts=128, drop=0.0, width=4096, dtype="bf16"),
        # A long batch, some slots dropped.
        dict(name="dispatch batch", op="dispatch", tokens=16384, slots=8, experts=64, drop=0.02, width=2048, dtype="bf16"),
        # Decoding: few rows per expert, all of the experts' weights are read.
        dict(name="matmul decode", op="matmul", rows=128, unused=0, experts=64, skew=1.0, inner=2048, outer=2048,
             dtype="bf16", act="silu", bias=True, residual=False, pre=False, quantize=False),
        # A short prompt through a narrow layer: ragged groups, widths that
        # are no multiple of a tile or of a block, the residual added.
        dict(name="matmul prompt ragged", op="matmul", rows=3001, unused=57, experts=8, skew=2.0, inner=1000,
             outer=1160, dtype="f16", act="relu", bias=True, residual=True, pre=False, quantize=False),
        # A long batch's first product, quantised again for the second.
        dict(name="matmul batch quantized", op="matmul", rows=16384, unused=100, experts=16, skew=1.0, inner=2048,
             outer=2048, dtype="bf16", act="silu", bias=True, residual=False, pre=False, quantize=True),
        # A training step's first product, keeping the values before the
        # activation for the gradient.
        dict(name="matmul train", op="matmul", rows=32768, unused=0, experts=16, skew=1.0, inner=2048, outer=4096,
             dtype="bf16", act="gelu", bias=True, residual=False, pre=True, quantize=False),
        # The norm before a block, 64 sequences being decoded: pure latency.
        dict(name="norm decode", op="norm", rows=64, width=4096, dtype="bf16", params="bf16", block=False, after=False,
             gate=0, scale=1.0),
        # Out of one block and into the next in a training step: the norm
        # after the block, a gate for each of 8 sequences, a residual scale.
        dict(name="norm train", op="norm", rows=16384, width=2048, dtype="bf16", params="f32", block=True, after=True,
             gate=8, scale=0.7),
        # Its gradient.
        dict(name="norm grad train", op="norm_grad", rows=16384, width=2048, dtype="bf16", params="f32", block=True,
             after=True, gate=8, scale=0.7, dy=True),
        # The gradient of a norm before a block in 32 bits, odd sizes.
        dict(name="norm grad odd", op="norm_grad", rows=4099, width=1037, dtype="f32", params="f32", block=False,
             after=False, gate=0, scale=1.0, dy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize_weights", "dispatch", "dispatch", "matmul", "matmul", "matmul", "norm", "norm",
                     "norm_grad", "norm_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "quantize_weights":
        outer, inner = _log(rng, 64, 4096), 8 * _log(rng, 8, 512)
        return dict(op=op, experts=_log(rng, 1, max(1, (1 << 27) // (outer * inner))), outer=outer, inner=inner, dtype=dtype,
                    transposed=rng.random() < 0.4)
    if op == "matmul":
        inner = rng.choice([16 * _log(rng, 8, 256), _log(rng, 100, 4096) | 1])
        outer = rng.choice([16 * _log(rng, 8, 256), 8 * _log(rng, 16, 512), _log(rng, 100, 4096) | 1])
        experts, quantize = rng.choice([1, 4, 8, 16, 32]), rng.random() < 0.35
        # no dearer than the largest listed product, plain form's padding included
        rows = _log(rng, 1, max(2, min(32768, (1 << 38) // (inner * outer))))
        return dict(op=op, rows=rows, unused=rng.choice([0, 0, rows // 10]), experts=experts,
                    skew=rng.choice([0.0, 1.0, 2.0]) if experts > 1 else 0.0, inner=inner, outer=outer,
                    dtype=rng.choice(["f16", "bf16"]), act=rng.choice(["none", "relu", "gelu", "silu"]),
                    bias=rng.random() < 0.7, residual=not quantize and rng.random() < 0.4, pre=rng.random() < 0.3,
                    quantize=quantize)
    width = rng.choice([8 * _log(rng, 8, 1024), _log(rng, 64, 8192) | 1])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 27) // width)), width=width, dtype=dtype)
    if op == "dispatch":
        slots = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, tokens=_log(rng, 1, min(131072, (1 << 28) // (slots * width))), slots=slots,
                    experts=max(slots, _log(rng, 8, 512)), drop=rng.choice([0.0, 0.0, 0.05, 0.5]), width=width, dtype=dtype)
    gate = rng.choice([-1, 0, 1, 4, 32])  # sequences with a gate of their own; 0: one for all, -1: none
    rows = _log(rng, 1, min(131072, (1 << 25) // width))
    rows = (rows + gate - 1) // gate * gate if gate > 1 else rows
    block = rng.random() < 0.7
    return dict(op=op, rows=rows, width=width, dtype=dtype, params=rng.choice(["f32", dtype]), block=block,
                after=block and rng.random() < 0.6, gate=gate if block else 0,
                scale=rng.choice([1.0, 0.7, 1.4142135]) if block else 1.0, dy=block or rng.random() < 0.7)


def _counts(case):
    """Rows per expert, largest first: proportional to exp(-skew * i / E), summing to the rows in use."""
    e, used = case["experts"], case["rows"] - case["unused"]
    share = [math.exp(-case["skew"] * i / e) for i in range(e)]
    edge, total, so_far = [0], sum(share), 0.0
    for s in share:
        so_far += s
        edge.append(min(used, int(round(used * so_far / total))))
    edge[-1] = used
    return [b - a for a, b in zip(edge, edge[1:])]


# ------------------------------------------------------------- plain forms

def _fit(amax):
    """Exponents of the scales for blocks of this largest magnitude: amax =
    m 2^e with 0.5 <= m < 1, and 448 = 0.875 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, e, 0).to(torch.int32)


def _power(e):
    """2^e in 32 bits, by its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _scales(e):
    return (e + 127).to(torch.uint8).view(E8M0)


def _quantize(x):
    r, w = x.shape
    n = -(-w // 128)
    v = torch.zeros(r, n * 128, device=x.device)
    v[:, :w] = x
    v = v.view(r, n, 128)
    e = _fit(v.abs().amax(2))
    q = (v * _power(-e)[..., None]).view(r, n * 128)[:, :w]
    return q.to(E4M3), _scales(e)


def _quantize_weights(w):
    e, n, k = w.shape
    bn, bk = -(-n // 128), -(-k // 128)
    v = torch.zeros(e, bn * 128, bk * 128, device=w.device)
    v[:, :n, :k] = w
    v = v.view(e, bn, 128, bk, 128)
    s = _fit(v.abs().amax((2, 4)))
    q = (v * _power(-s)[:, :, None, :, None]).view(e, bn * 128, bk * 128)[:, :n, :k]
    return q.to(E4M3), _scales(s)


def _aligned(q):
    """The same values with rows that start on 16 bytes, as the quantisers lay them out."""
    *lead, w = q.shape
    out = torch.zeros(*lead, (w + 15) // 16 * 16, dtype=torch.uint8, device=q.device)
    out[..., :w] = q.view(torch.uint8)
    return out.view(E4M3)[..., :w]


def _values(q, scales, blocks_down=False):
    """What quantised rows, or weights, stand for, in 32 bits."""
    s = scales.float().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if blocks_down:
        s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return q.float() * s


def _ids(case, gen):
    """Distinct experts per token from a skewed router; dropped slots are -1."""
    t, k, e = case["tokens"], case["slots"], case["experts"]
    score = torch.randn(t, e, device=DEVICE, generator=gen)
    score += 0.7 * torch.randn(e, device=DEVICE, generator=gen)
    ids = score.topk(k, dim=1).indices
    if case["drop"]:
        ids[torch.rand(t, k, device=DEVICE, generator=gen) < case["drop"]] = -1
    return ids


def _order(ids, experts):
    key = torch.where((ids < 0) | (ids >= experts), experts, ids).flatten().to(torch.int32)
    sorted_key, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    edges = torch.arange(experts + 1, device=order.device, dtype=torch.int32)
    offsets = torch.searchsorted(sorted_key, edges)
    return position.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op = case["op"]
    state = dict(case=case, op=op)

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, device=DEVICE, generator=gen) * scale).to(dtype or DTYPES[case["dtype"]])

    def stream(rows, width):
        """Rows as a residual stream has them: channels and tokens of different sizes."""
        x = torch.randn(rows, width, device=DEVICE, generator=gen)
        x *= torch.exp(0.8 * torch.randn(width, device=DEVICE, generator=gen))
        x *= torch.exp(0.5 * torch.randn(rows, 1, device=DEVICE, generator=gen))
        return x.to(DTYPES[case["dtype"]])

    if op == "quantize":
        state["x"] = stream(case["rows"], case["width"])
    elif op == "quantize_weights":
        e, n, k = case["experts"], case["outer"], case["inner"]
        w = normal(e, k, n, scale=k ** -0.5).transpose(1, 2) if case["transposed"] else normal(e, n, k, scale=k ** -0.5)
        state["w"] = w
    elif op == "dispatch":
        state["position"], state["offsets"] = _order(_ids(case, gen), case["experts"])
        state["x"] = stream(case["tokens"], case["width"])
    elif op == "matmul":
        rows, e, n, k = case["rows"], case["experts"], case["outer"], case["inner"]
        counts = _counts(case)
        state["most"] = max(counts)  # the largest group: a program's capacity
        random.Random(seed).shuffle(counts)
        edges = [0]
        for c in counts:
            edges.append(edges[-1] + c)
        state["offsets"] = torch.tensor(edges, dtype=torch.int32).to(DEVICE)
        q, state["xs"] = _quantize(stream(rows, k))
        state["x"] = _aligned(q)
        q, state["ws"] = _quantize_weights(normal(e, n, k, scale=k ** -0.5))
        state["w"] = _aligned(q)
        state["bias"] = normal(e, n, scale=0.5) if case["bias"] else None
        state["residual"] = normal(rows, n) if case["residual"] else None
    else:
        rows, width, params = case["rows"], case["width"], DTYPES[case["params"]]

        def weight():
            return (1.0 + normal(width, scale=0.2, dtype=torch.float32)).to(params)

        state["x"], state["weight"] = stream(rows, width), weight()
        state["block"] = normal(rows, width, scale=0.5) if case["block"] else None
        state["after"] = weight() if case["after"] else None
        groups = case["gate"]
        shape = (width,) if groups == 0 else (groups, width)
        state["gate"] = normal(*shape, scale=0.5, dtype=params) if case["block"] and groups >= 0 else None
        if op == "norm_grad":
            state["dh"] = normal(rows, width, scale=0.1)
            state["dy"] = normal(rows, width, scale=0.1) if case["dy"] else None
    return state


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_matmul(s):
    c = s["case"]
    rows, start = c["rows"], s["offsets"].long()
    step = torch.arange(s["most"], device=DEVICE)
    at, real = start[:-1, None] + step, step < (start[1:] - start[:-1])[:, None]
    xp = _values(s["x"], s["xs"])[at.clamp(max=rows - 1)] * real[..., None]
    z = torch.bmm(xp, _values(s["w"], s["ws"], True).transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None]
    row = torch.arange(rows, device=DEVICE)
    expert = (torch.searchsorted(start, row, right=True) - 1).clamp(0, c["experts"] - 1)
    inside = (row < start[-1])[:, None]
    at = (expert * s["most"] + row - start[expert]).clamp(0, c["experts"] * s["most"] - 1)
    z = torch.where(inside, z.flatten(0, 1)[at], torch.zeros((), device=DEVICE))
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = torch.where(inside, y + s["residual"].float(), y)
    out = {}
    if c["quantize"]:
        out["q"], out["scales"] = _quantize(y)
    else:
        out["y"] = y.to(DTYPES[c["dtype"]])
    if c["pre"]:
        out["z"] = z.to(DTYPES[c["dtype"]])
    return out


def _root(v):
    return 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)


def _gates(gate, rows):
    """The gate of each row, broadcast."""
    if gate is None or gate.dim() == 1:
        return 1.0 if gate is None else gate.float()
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _plain_join(s):
    """y in 32 bits, as it is held."""
    if s["block"] is None:
        return s["x"].float()
    b = s["block"].float()
    u = b if s["after"] is None else b * _root(b) * s["after"].float()
    y = s["case"]["scale"] * s["x"].float() + _gates(s["gate"], b.shape[0]) * u
    return y.to(s["x"].dtype).float()


def _norm_back(d, v, weight):
    """The gradients of v * _root(v) * weight for v and weight."""
    r = _root(v)
    n, g = v * r, d * weight.float()
    return r * (g - n * (g * n).mean(1, keepdim=True)), (d * n).sum(0)


def _plain_norm_grad(s):
    y, dtype, rows = s["x"].float(), s["x"].dtype, s["x"].shape[0]  # the state's x stands for y here
    dx, dweight = _norm_back(s["dh"].float(), y, s["weight"])
    if s["dy"] is not None:
        dx = dx + s["dy"].float()
    out = {"dx": (s["case"]["scale"] * dx).to(dtype), "dweight": dweight.to(s["weight"].dtype)}
    if s["block"] is None:
        return out
    b, gate = s["block"].float(), s["gate"]
    u = b if s["after"] is None else b * _root(b) * s["after"].float()
    if gate is not None:
        part = (dx * u).view(1 if gate.dim() == 1 else gate.shape[0], -1, u.shape[1]).sum(1)
        out["dgate"] = part.view(gate.shape).to(gate.dtype)
    du = dx * _gates(gate, rows)
    if s["after"] is not None:
        du, dafter = _norm_back(du, b, s["after"])
        out["dafter"] = dafter.to(s["after"].dtype)
    out["dblock"] = du.to(dtype)
    return out


def _plain(s):
    op = s["op"]
    if op == "quantize":
        q, scales = _quantize(s["x"])
        return {"q": q, "scales": scales}
    if op == "quantize_weights":
        q, scales = _quantize_weights(s["w"])
        return {"q": q, "scales": scales}
    if op == "dispatch":
        q, scales = _quantize(s["x"])
        t, k = s["position"].shape
        token = torch.empty(t * k, dtype=torch.int64, device=DEVICE)
        token[s["position"].flatten().long()] = torch.arange(t * k, device=DEVICE) // k
        kept = torch.arange(t * k, device=DEVICE)[:, None] < s["offsets"][-1]
        zero = torch.zeros((), dtype=torch.uint8, device=DEVICE)
        return {"q": torch.where(kept, q.view(torch.uint8)[token], zero).view(E4M3),
                "scales": torch.where(kept, scales.view(torch.uint8)[token], zero + 127).view(E8M0)}
    if op == "matmul":
        return _plain_matmul(s)
    if op == "norm":
        y = _plain_join(s)
        h = (y * _root(y) * s["weight"].float()).to(s["x"].dtype)
        return {"h": h} if s["block"] is None else {"y": y.to(s["x"].dtype), "h": h}
    return _plain_norm_grad(s)


def run(state):
    if not own:
        return _plain(state)
    import lsd_radix_sort_key_gb300 as rs
    s, op, case = state, state["op"], state["case"]
    if op == "quantize":
        q, scales = rs.expert_quantize(s["x"])
        return {"q": q, "scales": scales}
    if op == "quantize_weights":
        q, scales = rs.expert_quantize_weights(s["w"])
        return {"q": q, "scales": scales}
    if op == "dispatch":
        q, scales = rs.expert_dispatch_quantized(s["x"], s["position"], s["offsets"])
        return {"q": q, "scales": scales}
    if op == "matmul":
        got = rs.expert_matmul_quantized(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], bias=s["bias"],
                                         activation=case["act"], residual=s["residual"], dtype=DTYPES[case["dtype"]],
                                         return_pre=case["pre"], quantize=case["quantize"])
        if not case["pre"] and not case["quantize"]:
            return {"y": got}
        out = {"q": got[0], "scales": got[1]} if case["quantize"] else {"y": got[0]}
        if case["pre"]:
            out["z"] = got[-1]
        return out
    if op == "norm":
        if s["block"] is None:
            return {"h": rs.expert_norm(s["x"], s["weight"], eps=EPS)}
        y, h = rs.expert_norm(s["x"], s["weight"], block=s["block"], block_weight=s["after"], gate=s["gate"],
                              residual_scale=case["scale"], eps=EPS)
        return {"y": y, "h": h}
    dx, dweight, dblock, dafter, dgate = rs.expert_norm_grad(s["dh"], s["x"], s["weight"], dy=s["dy"], block=s["block"],
                                                             block_weight=s["after"], gate=s["gate"],
                                                             residual_scale=case["scale"], eps=EPS)
    out = {"dx": dx, "dweight": dweight}
    if dblock is not None:
        out["dblock"] = dblock
    if dafter is not None:
        out["dafter"] = dafter
    if dgate is not None:
        out["dgate"] = dgate
    return out


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "quantize":
        n = case["rows"] * case["width"]
        return {"bytes": n * (size + 1) + case["rows"] * -(-case["width"] // 128), "flops": 0}
    if op == "quantize_weights":
        n = case["experts"] * case["outer"] * case["inner"]
        return {"bytes": n * (size + 1) + case["experts"] * -(-case["outer"] // 128) * -(-case["inner"] // 128), "flops": 0}
    if op == "dispatch":
        t, k, h = case["tokens"], case["slots"], case["width"]
        return {"bytes": t * h * size + t * k * (h + -(-h // 128)) + 4 * t * k, "flops": 0}
    if op == "matmul":
        rows, used, n, k = case["rows"], case["rows"] - case["unused"], case["outer"], case["inner"]
        active = sum(c > 0 for c in _counts(case))
        moved = used * k + active * n * k + (used + active * -(-n // 128)) * -(-k // 128)
        moved += rows * (n + -(-n // 128)) if case["quantize"] else 2 * rows * n
        moved += 2 * (rows * n * case["pre"] + active * n * case["bias"] + used * n * case["residual"])
        return {"bytes": moved, "flops": 2 * used * n * k}
    rows, width = case["rows"], case["width"]
    gate = case["gate"] if case["block"] else -1
    params = (1 + case["after"] + (0 if gate < 0 else max(1, gate))) * width * (4 if case["params"] == "f32" else 2)
    if op == "norm":
        return {"bytes": rows * width * size * (4 if case["block"] else 2) + params,
                "flops": rows * width * (4 + 3 * case["block"] + 4 * case["after"])}
    read = 2 + case["dy"] + case["block"]
    return {"bytes": rows * width * size * (read + 1 + case["block"]) + 2 * params,
            "flops": rows * width * (10 + 4 * case["block"] + 10 * case["after"])}


# ------------------------------------------------------------ definitions

def _round_e4m3(v):
    """Values of magnitude up to 448 to the nearest with three bits after the
    leading one, ties to even, in steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _nearest(v, down=1):
    """v [rows, width] in blocks of `down` rows and 128 columns: (e4m3 values, scales) in 64 bits."""
    r, w = v.shape
    n, m = -(-w // 128), -(-r // down)
    q, scales = torch.empty_like(v), torch.empty(m, n, dtype=torch.float64, device=v.device)
    for j in range(n):
        part = v[:, j * 128:(j + 1) * 128]
        largest = torch.zeros(m * down, dtype=torch.float64, device=v.device)
        largest[:r] = part.abs().max(1).values
        largest = largest.view(m, down).max(1).values
        s = torch.exp2(torch.floor(torch.log2(largest.clamp(min=1e-300) / 448)).clamp(min=-126))
        s = torch.where(largest > 448 * s, 2 * s, s)
        s = torch.where(largest > 0, s, torch.ones_like(s))
        scales[:, j] = s
        q[:, j * 128:(j + 1) * 128] = _round_e4m3(part / s.repeat_interleave(down)[:r, None])
    return q, scales


def exact(case, seed):
    """The operators in 64 bits, expert by expert and block by block."""
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        q, scales = _nearest(s["x"].double())
        return {"q": q, "scales": scales}
    if op == "quantize_weights":
        done = [_nearest(w.double(), 128) for w in s["w"]]
        return {"q": torch.stack([q for q, _ in done]), "scales": torch.stack([t for _, t in done])}
    if op == "dispatch":
        t, k = s["position"].shape
        q, scales = _nearest(s["x"].double())
        rows = torch.zeros(t * k, q.shape[1], dtype=torch.float64, device=DEVICE)
        rows_scales = torch.ones(t * k, scales.shape[1], dtype=torch.float64, device=DEVICE)
        for j in range(k):
            at = s["position"][:, j].long()
            sent = at < s["offsets"][-1]
            rows[at[sent]], rows_scales[at[sent]] = q[sent], scales[sent]
        return {"q": rows, "scales": rows_scales}
    if op == "matmul":
        rows, n, k, act = case["rows"], case["outer"], case["inner"], case["act"]
        y, z = (torch.zeros(rows, n, dtype=torch.float64, device=DEVICE) for _ in range(2))
        edges = s["offsets"].tolist()
        for e, (a, b) in enumerate(zip(edges, edges[1:])):
            if a == b:
                continue
            part = torch.zeros(b - a, n, dtype=torch.float64, device=DEVICE)
            for j in range(0, k, 128):
                xj = s["x"][a:b, j:j + 128].double() * s["xs"][a:b, j // 128, None].double()
                wj = s["w"][e, :, j:j + 128].double() * s["ws"][e, :, j // 128].double().repeat_interleave(128)[:n, None]
                part += xj @ wj.T
            if s["bias"] is not None:
                part += s["bias"][e].double()
            z[a:b] = part
            if act == "relu":
                part = part.clamp(min=0)
            elif act == "gelu":
                part = part * torch.special.ndtr(part)
            elif act == "silu":
                part = part * torch.sigmoid(part)
            y[a:b] = part if s["residual"] is None else part + s["residual"][a:b].double()
        out = {"y": y}
        if case["quantize"]:
            q, scales = _nearest(y)
            out = {"q": q, "scales": scales}
        if case["pre"]:
            out["z"] = z
        return out

    def inverse_rms(v):
        return torch.rsqrt(torch.linalg.vecdot(v, v) / v.shape[1] + EPS)[:, None]

    x, weight, block = s["x"].double(), s["weight"].double(), s["block"]
    rows, width = x.shape
    b = None if block is None else block.double()
    gate = None if s["gate"] is None else s["gate"].double()
    per_row = None if gate is None else gate.expand(rows, width) if gate.dim() == 1 else (
        gate[torch.arange(rows, device=DEVICE) * gate.shape[0] // rows])
    u = None if b is None else b if s["after"] is None else b * inverse_rms(b) * s["after"].double()
    if op == "norm":
        y = x
        if b is not None:
            y = case["scale"] * x + (u if per_row is None else per_row * u)
        held = y.to(s["x"].dtype).double()  # the norm is of y as it is held
        h = held * inverse_rms(held) * weight
        return {"h": h} if b is None else {"y": y, "h": h}

    def back(d, v, w):
        # d(v_i r)/dv_j = r (i == j) - v_i v_j r^3 / width
        r, g = inverse_rms(v), d * w
        return g * r - v * r ** 3 * (torch.linalg.vecdot(g, v) / width)[:, None], (d * v * r).sum(0)

    dx, dweight = back(s["dh"].double(), x, weight)
    if s["dy"] is not None:
        dx = dx + s["dy"].double()
    out = {"dx": case["scale"] * dx, "dweight": dweight}
    if b is None:
        return out
    if gate is not None:
        out["dgate"] = (dx * u).sum(0) if gate.dim() == 1 else (dx * u).unflatten(0, (gate.shape[0], -1)).sum(1)
    du = dx if per_row is None else dx * per_row
    if s["after"] is not None:
        du, out["dafter"] = back(du, b, s["after"].double())
    out["dblock"] = du
    return out
