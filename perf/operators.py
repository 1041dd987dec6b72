"""Workloads of the expert operators: tokens sorted by expert, rows sent to
their experts and back, and the experts' products.

A mixture-of-experts layer gives each of T tokens K of E experts.  The
operators here are the steps between the router's choice and the layer's
output, and their gradients:

  sort      expert numbers [T, K] -> the stable order of the T*K slots by
            expert, its inverse and the experts' row ranges.  A number outside
            [0, E) is a dropped slot; those come last.
  dispatch  the tokens' rows laid out by expert (dropped slots: zero rows),
            and its gradient (each token's sum over its slots).
  combine   each token's weighted sum of its experts' rows, and its gradient
            for the rows and for the weights.
  matmul    per expert: activation(x w^T + bias) + residual, rows past the
            last expert's zero, and its gradient for x, w and bias.

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


def listed():
    return [
        # One decoding step of 64 sequences: the sort is pure latency.
        dict(name="sort decode", op="sort", tokens=64, slots=8, experts=128, drop=0.0, ids="i64"),
        # A prompt on one of several machines: an odd token count, and the
        # slots of experts that live elsewhere are dropped (-1).
        dict(name="sort prompt odd", op="sort", tokens=5003, slots=6, experts=160, drop=0.25, ids="i32"),
        # A training batch: a million slots.
        dict(name="sort train", op="sort", tokens=131072, slots=8, experts=256, drop=0.0, ids="i64"),
        # A prompt's rows sent to their experts; an odd token count, a width
        # that is no multiple of 64, dropped slots.
        dict(name="dispatch prompt", op="dispatch", tokens=4099, slots=4, experts=64, drop=0.02, width=1032, dtype="f16"),
        # The gradient of the dispatch in a training step.
        dict(name="dispatch grad train", op="dispatch_grad", tokens=16384, slots=8, experts=64, drop=0.0, width=2048,
             dtype="bf16"),
        # The way back for a few sequences that are being decoded.
        dict(name="combine decode", op="combine", tokens=8, slots=8, experts=128, drop=0.0, width=4096, dtype="bf16"),
        # The way back in a training step.
        dict(name="combine train", op="combine", tokens=16384, slots=8, experts=64, drop=0.0, width=2048, dtype="bf16"),
        # Its gradient, rows and weights, for a model trained in 32 bits with
        # a capacity limit that dropped some slots.
        dict(name="combine grad train", op="combine_grad", tokens=8191, slots=2, experts=16, drop=0.05, width=4096,
             dtype="f32"),
        # Decoding: few rows per expert, all of the experts' weights are read.
        dict(name="matmul decode", op="matmul", rows=128, unused=0, experts=64, skew=1.0, inner=2048, outer=2048,
             dtype="bf16", act="silu", bias=True, residual=False, pre=False),
        # A short prompt through a narrow layer: ragged groups, widths that
        # are no multiple of a tile, the residual added in the product.
        dict(name="matmul prompt ragged", op="matmul", rows=3001, unused=57, experts=8, skew=2.0, inner=1000,
             outer=1160, dtype="f16", act="relu", bias=True, residual=True, pre=False),
        # A training step's first expert product, keeping the values before
        # the activation for the gradient.
        dict(name="matmul train", op="matmul", rows=32768, unused=0, experts=16, skew=1.0, inner=2048, outer=4096,
             dtype="bf16", act="gelu", bias=True, residual=False, pre=True),
        # The gradient of such a product.
        dict(name="matmul grad train", op="matmul_grad", rows=16384, unused=100, experts=16, skew=1.0, inner=2048,
             outer=2048, dtype="bf16", act="silu", bias=True, residual=False, pre=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch_grad", "combine", "combine_grad", "matmul", "matmul", "matmul_grad"])
    if op == "sort":
        slots = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, tokens=_log(rng, 1, (1 << 20) // slots), slots=slots, experts=max(slots, _log(rng, 8, 512)),
                    drop=rng.choice([0.0, 0.0, 0.05, 0.5]), ids=rng.choice(["i32", "i64"]))
    if not op.startswith("matmul"):
        slots = rng.choice([1, 2, 4, 6, 8])
        width = rng.choice([8 * _log(rng, 8, 1024), _log(rng, 64, 8192) | 1])
        most = min(131072, (1 << 28) // (slots * width))
        return dict(op=op, tokens=_log(rng, 1, most), slots=slots, experts=max(slots, _log(rng, 8, 512)),
                    drop=rng.choice([0.0, 0.0, 0.05, 0.5]), width=width, dtype=rng.choice(["f32", "f16", "bf16"]))
    inner, outer = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512)
    experts = rng.choice([1, 4, 8, 16, 32])
    products = 1 if op == "matmul" else 2
    # no dearer than the largest listed product, plain form's padding included
    most = min(32768, (1 << 38) // (products * inner * outer))
    rows = _log(rng, 1, max(2, most))
    return dict(op=op, rows=rows, unused=rng.choice([0, 0, rows // 10]), experts=experts,
                skew=rng.choice([0.0, 1.0, 2.0]) if experts > 1 else 0.0, inner=inner, outer=outer,
                dtype=rng.choice(["f16", "bf16"]), act=rng.choice(["none", "relu", "gelu", "silu"]),
                bias=rng.random() < 0.7, residual=op == "matmul" and rng.random() < 0.4, pre=op != "matmul" or rng.random() < 0.3)


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
    return order.to(torch.int32), position.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    state = dict(case=case, op=case["op"])

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, device=DEVICE, generator=gen) * scale).to(dtype or DTYPES[case["dtype"]])

    if case["op"] == "sort":
        state["ids"] = _ids(case, gen).to(torch.int32 if case["ids"] == "i32" else torch.int64)
        return state
    if not case["op"].startswith("matmul"):
        t, k, h = case["tokens"], case["slots"], case["width"]
        _, state["position"], state["offsets"] = _order(_ids(case, gen), case["experts"])
        if case["op"] == "dispatch":
            state["x"] = normal(t, h)
        if case["op"] in ("dispatch_grad", "combine", "combine_grad"):
            state["y"] = normal(t * k, h)
        if case["op"] in ("combine", "combine_grad"):
            state["weights"] = torch.softmax(torch.randn(t, k, device=DEVICE, generator=gen), dim=1)
        if case["op"] == "combine_grad":
            state["dout"] = normal(t, h, scale=0.1)
        return state
    rows, e, n, k = case["rows"], case["experts"], case["outer"], case["inner"]
    counts = _counts(case)
    state["most"] = max(counts)  # the largest group: a program's capacity
    random.Random(seed).shuffle(counts)
    edges = [0]
    for c in counts:
        edges.append(edges[-1] + c)
    state["offsets"] = torch.tensor(edges, dtype=torch.int32).to(DEVICE)
    state["x"] = normal(rows, k)
    state["w"] = normal(e, n, k, scale=k ** -0.5)
    state["bias"] = normal(e, n, scale=0.5) if case["bias"] else None
    state["residual"] = normal(rows, n) if case["residual"] else None
    if case["op"] == "matmul_grad":
        state["dy"] = normal(rows, n, scale=0.1)
        state["z"] = normal(rows, n) if case["act"] != "none" else None
    return state


# ------------------------------------------------------------- plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.7071067811865476))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _padded(s, rows):
    """Row numbers [E, most] of each expert's rows, and which of them are real."""
    start = s["offsets"].long()
    step = torch.arange(s["most"], device=DEVICE)
    at = start[:-1, None] + step
    real = step < (start[1:] - start[:-1])[:, None]
    return at.clamp(max=rows - 1), real


def _unpadded(s, groups, rows):
    """[E, most, width] -> [rows, width], zero past the last expert's rows."""
    start, row = s["offsets"].long(), torch.arange(rows, device=DEVICE)
    expert = (torch.searchsorted(start, row, right=True) - 1).clamp(0, s["case"]["experts"] - 1)
    inside = (row < start[-1])[:, None]
    at = (expert * s["most"] + row - start[expert]).clamp(0, groups.shape[0] * groups.shape[1] - 1)
    return torch.where(inside, groups.flatten(0, 1)[at], torch.zeros((), device=DEVICE))


def _plain_matmul(s):
    c, x = s["case"], s["x"]
    at, real = _padded(s, c["rows"])
    xp = x.float()[at] * real[..., None]
    z = torch.bmm(xp, s["w"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None]
    z = _unpadded(s, z, c["rows"])
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = torch.where(torch.arange(c["rows"], device=DEVICE)[:, None] < s["offsets"][-1], y + s["residual"].float(), y)
    y = y.to(x.dtype)
    return {"y": y, "z": z.to(x.dtype)} if c["pre"] else y


def _plain_matmul_grad(s):
    c, x = s["case"], s["x"]
    at, real = _padded(s, c["rows"])
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), c["act"])
    dzp = dz[at] * real[..., None]
    xp = x.float()[at] * real[..., None]
    dx = _unpadded(s, torch.bmm(dzp, s["w"].float()), c["rows"]).to(x.dtype)
    dw = torch.bmm(dzp.transpose(1, 2), xp).to(x.dtype)
    out = {"dx": dx, "dw": dw}
    if s["bias"] is not None:
        out["dbias"] = dzp.sum(1).to(x.dtype)
    return out


def _rows_of(s):
    """[T, K, width] of y in 32 bits, zero for dropped slots."""
    position = s["position"].long()
    kept = (position < s["offsets"][-1])[..., None]
    return torch.where(kept, s["y"][position].float(), torch.zeros((), device=DEVICE)), kept


def _plain(s):
    op = s["op"]
    if op == "sort":
        order, position, offsets = _order(s["ids"], s["case"]["experts"])
        return {"order": order, "position": position, "offsets": offsets}
    if op == "dispatch":
        t, k = s["position"].shape
        token = torch.empty(t * k, dtype=torch.int64, device=DEVICE)
        token[s["position"].flatten().long()] = torch.arange(t * k, device=DEVICE) // k
        kept = torch.arange(t * k, device=DEVICE)[:, None] < s["offsets"][-1]
        return torch.where(kept, s["x"][token], torch.zeros((), dtype=s["x"].dtype, device=DEVICE))
    if op == "dispatch_grad":
        return _rows_of(s)[0].sum(1).to(s["y"].dtype)
    if op == "combine":
        return (_rows_of(s)[0] * s["weights"][..., None]).sum(1).to(s["y"].dtype)
    if op == "combine_grad":
        rows, kept = _rows_of(s)
        dout = s["dout"].float()[:, None]
        dy = torch.empty_like(s["y"])
        scaled = torch.where(kept, dout * s["weights"][..., None], torch.zeros((), device=DEVICE))
        dy[s["position"].flatten().long()] = scaled.to(dy.dtype).flatten(0, 1)
        return {"dy": dy, "dweights": (rows * dout).sum(2)}
    return _plain_matmul(s) if op == "matmul" else _plain_matmul_grad(s)


def run(state):
    if not own:
        return _plain(state)
    import lsd_radix_sort_key_gb300 as rs
    op, case = state["op"], state["case"]
    if op == "sort":
        order, position, offsets = rs.expert_sort(state["ids"], case["experts"])
        return {"order": order, "position": position, "offsets": offsets}
    if op == "dispatch":
        return rs.expert_dispatch(state["x"], state["position"], state["offsets"])
    if op == "dispatch_grad":
        return rs.expert_dispatch_grad(state["y"], state["position"], state["offsets"])
    if op == "combine":
        return rs.expert_combine(state["y"], state["weights"], state["position"], state["offsets"])
    if op == "combine_grad":
        dy, dweights = rs.expert_combine_grad(state["dout"], state["y"], state["weights"], state["position"], state["offsets"])
        return {"dy": dy, "dweights": dweights}
    if op == "matmul":
        if case["pre"]:
            y, z = rs.expert_matmul(state["x"], state["w"], state["offsets"], bias=state["bias"], activation=case["act"],
                                    residual=state["residual"], return_pre=True)
            return {"y": y, "z": z}
        return rs.expert_matmul(state["x"], state["w"], state["offsets"], bias=state["bias"], activation=case["act"],
                                residual=state["residual"])
    dx, dw, dbias = rs.expert_matmul_grad(state["dy"], state["x"], state["w"], state["offsets"], pre=state["z"],
                                          activation=case["act"], bias=state["bias"] is not None)
    out = {"dx": dx, "dw": dw}
    if dbias is not None:
        out["dbias"] = dbias
    return out


def work(case):
    op = case["op"]
    if op == "sort":
        n = case["tokens"] * case["slots"]
        return {"bytes": n * ((4 if case["ids"] == "i32" else 8) + 8) + 4 * (case["experts"] + 1), "flops": 0}
    if not op.startswith("matmul"):
        t, k, h = case["tokens"], case["slots"], case["width"]
        row = h * (4 if case["dtype"] == "f32" else 2)
        kept = 1.0 - case["drop"]
        plan = 4 * t * k
        if op == "dispatch":
            return {"bytes": (t + t * k) * row + plan, "flops": 0}
        if op == "dispatch_grad":
            return {"bytes": (t + t * k * kept) * row + plan, "flops": t * k * kept * h}
        if op == "combine":
            return {"bytes": (t + t * k * kept) * row + plan + 4 * t * k, "flops": 2 * t * k * kept * h}
        return {"bytes": (t + t * k * (1 + kept)) * row + plan + 8 * t * k, "flops": 3 * t * k * kept * h}
    rows, used, n, k = case["rows"], case["rows"] - case["unused"], case["outer"], case["inner"]
    active = sum(c > 0 for c in _counts(case))
    weights = active * n * k + (active * n if case["bias"] else 0)
    if op == "matmul":
        moved = used * k + weights + rows * n * (1 + case["pre"]) + (used * n if case["residual"] else 0)
        return {"bytes": 2 * moved, "flops": 2 * used * n * k}
    moved = used * n * (2 if case["act"] != "none" else 1) + used * k + active * n * k
    moved += rows * k + case["experts"] * n * (k + bool(case["bias"]))
    return {"bytes": 2 * moved, "flops": 4 * used * n * k}


# ------------------------------------------------------------ definitions

def exact(case, seed):
    """The operators in 64 bits, expert by expert and slot by slot."""
    if case["op"] == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    last = int(s["offsets"][-1])
    if not case["op"].startswith("matmul"):
        t, k, h = case["tokens"], case["slots"], case["width"]
        if case["op"] == "dispatch":
            out = torch.zeros(t * k, h, dtype=torch.float64, device=DEVICE)
            for j in range(k):
                at = s["position"][:, j].long()
                sent = at < last
                out[at[sent]] = s["x"][sent].double()
            return out
        grad = case["op"] == "combine_grad"
        out = torch.zeros((t * k, h) if grad else (t, h), dtype=torch.float64, device=DEVICE)
        dweights = torch.zeros(t, k, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            at = s["position"][:, j].long()
            token = torch.nonzero(at < last).flatten()
            at = at[token]
            row = s["y"][at].double()
            if case["op"] == "dispatch_grad":
                out[token] += row
            elif case["op"] == "combine":
                out[token] += s["weights"][token, j, None].double() * row
            else:
                d = s["dout"][token].double()
                out[at] = s["weights"][token, j, None].double() * d
                dweights[token, j] = torch.linalg.vecdot(row, d)
        return {"dy": out, "dweights": dweights} if grad else out
    edges = s["offsets"].tolist()
    rows, n, k, act = case["rows"], case["outer"], case["inner"], case["act"]
    if case["op"] == "matmul":
        y = torch.zeros(rows, n, dtype=torch.float64, device=DEVICE)
        z = torch.zeros_like(y)
        for e, (a, b) in enumerate(zip(edges, edges[1:])):
            if a == b:
                continue
            part = torch.einsum("rk,nk->rn", s["x"][a:b].double(), s["w"][e].double())
            part = part if s["bias"] is None else part + s["bias"][e].double()
            z[a:b] = part
            if act == "relu":
                part = part.clamp(min=0)
            elif act == "gelu":
                part = part * torch.special.ndtr(part)
            elif act == "silu":
                part = part * torch.sigmoid(part)
            y[a:b] = part if s["residual"] is None else part + s["residual"][a:b].double()
        return {"y": y, "z": z} if case["pre"] else y
    dx = torch.zeros(rows, k, dtype=torch.float64, device=DEVICE)
    dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device=DEVICE)
    dbias = torch.zeros(case["experts"], n, dtype=torch.float64, device=DEVICE)
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        dz = s["dy"][a:b].double()
        if act != "none":
            z = s["z"][a:b].double()
            if act == "relu":
                dz = dz.masked_fill(z <= 0, 0.0)
            elif act == "gelu":
                dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi))
            else:
                g = torch.sigmoid(z)
                dz = dz * g * (1 + z - z * g)
        dx[a:b] = dz @ s["w"][e].double()
        dw[e] = dz.T @ s["x"][a:b].double()
        dbias[e] = dz.sum(0)
    out = {"dx": dx, "dw": dw}
    if s["bias"] is not None:
        out["dbias"] = dbias
    return out
