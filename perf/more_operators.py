"""The measured cases of what surrounds the library's expert layer: rows sorted by expert and joined again, layer norm,
products in 8-bit integers, and gradient clipping.

Operators (the public names of tile_size_selection_amd):
  sort_by_expert, gather_rows       a stable order of the router's choices by expert, and the tokens' rows in that order
  combine_rows, .._backward,        each token's weighted sum over its choices' rows, the gradients of rows and weights, and
    gather_rows_backward            the sum of its rows' gradients
  layer_norm, layer_norm_backward   layer norm of x + residual; gradients of x (= of the residual), weight and bias
  quantize_int8, gemm_int8          int8 with a scale for each row, and C = (A sa) (B sb)^T with scales for tokens and channels
  clip_grad_norm                    the norm over many tensors, and the tensors scaled to at most a given norm

A choice outside 0 .. experts - 1 is dropped: its place is behind all routed rows, written as the complement (~place) in
`row`, and its choice as the complement in `choice`; the rows there are zero, and nothing reads them.
Where `own` is false, run() computes the same from elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

EPS = 1e-5
SMALLEST_AMAX = 1e-30  # a row's largest magnitude is taken as at least this, so that its scale has a reciprocal
NORM_EPS = 1e-6        # added to the norm that a clip divides by
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---- the cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step on its way to its experts: latency is all that counts
        {"name": "dispatch_one_token", "op": "dispatch", "tokens": 1, "top": 8, "experts": 64, "d": 2048,
         "dtype": "bf16", "dropped": 0.0, "skew": 0.5},
        # a long prompt's quantised rows with their scales, eight experts a token
        {"name": "dispatch_prompt_fp8", "op": "dispatch", "tokens": 16384, "top": 8, "experts": 128, "d": 4096,
         "dtype": "e4m3", "dropped": 0.0, "skew": 1.0},
        # the end of an expert layer's forward pass, with choices that a capacity dropped and an odd number of tokens
        {"name": "combine_forward", "op": "combine", "tokens": 5001, "top": 6, "experts": 160, "d": 5120,
         "dtype": "bf16", "dropped": 0.05, "skew": 0.5},
        # the same layer's gradients: of the experts' rows, of the router's weights, and of the tokens
        {"name": "combine_backward", "op": "combine_backward", "tokens": 8200, "top": 4, "experts": 60, "d": 2048,
         "dtype": "f16", "dropped": 0.05, "skew": 0.5},
        # the norm of one token in a decode step
        {"name": "layer_norm_one_token", "op": "layer_norm", "rows": 1, "d": 4096, "dtype": "bf16", "residual": True},
        # norms of narrow rows: every head of every token of a batch
        {"name": "layer_norm_heads", "op": "layer_norm", "rows": 300000, "d": 128, "dtype": "f16", "residual": False},
        # the backward pass of a training step's norm
        {"name": "layer_norm_backward_train", "op": "layer_norm_backward", "rows": 16384, "d": 4096, "dtype": "bf16"},
        # a few sequences' decode step through a square projection, quantised on the way: the weights' bytes are the cost
        {"name": "int8_linear_decode", "op": "int8_linear", "m": 4, "n": 8192, "k": 8192, "dtype": "bf16"},
        # a prompt through a narrow projection, ragged tiles on both edges
        {"name": "int8_linear_prompt", "op": "int8_linear", "m": 3000, "n": 5000, "k": 2048, "dtype": "f16"},
        # a large batch through a square projection: the matrix cores are the cost
        {"name": "gemm_int8_8192", "op": "gemm_int8", "m": 8192, "n": 8192, "k": 8192, "out": "bf16"},
        # the small parameters of one layer: latency
        {"name": "clip_small", "op": "clip", "tensors": 12, "largest": 5120, "shapes": 1, "dtype": "f32", "ratio": 0.5},
        # a model's gradients, norms' weights and matrices of every size
        {"name": "clip_model", "op": "clip", "tensors": 60, "largest": 1 << 25, "shapes": 2, "dtype": "mixed",
         "ratio": 0.5},
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "combine", "combine_backward", "layer_norm", "layer_norm_backward",
                     "int8_linear", "int8_linear", "gemm_int8", "clip"])
    if op in ("dispatch", "combine", "combine_backward"):
        dtype = rng.choice(["bf16", "f16", "f32"] + (["e4m3"] if op == "dispatch" else []))
        d, top = _log_int(rng, 256, 8192, 8), rng.randint(1, 8)
        tokens = max(1, min(_log_int(rng, 1, 16384), (1 << 28) // (top * d * SIZE[dtype])))
        return {"op": op, "tokens": tokens, "top": top, "experts": _log_int(rng, max(2, top), 256), "d": d,
                "dtype": dtype, "dropped": rng.choice([0.0, 0.0, 0.05, 0.3]), "skew": rng.choice([0.0, 0.5, 1.0])}
    if op in ("layer_norm", "layer_norm_backward"):
        d = _log_int(rng, 64, 16384, 8)
        rows = min(_log_int(rng, 1, 300000), (1 << 26) // d)
        case = {"op": op, "rows": rows, "d": d, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
        if op == "layer_norm":
            case["residual"] = rng.random() < 0.5
        return case
    if op in ("int8_linear", "gemm_int8"):
        case = {"op": op, "m": _log_int(rng, 1, 8192), "n": _log_int(rng, 256, 8192), "k": _log_int(rng, 512, 8192, 16)}
        if op == "int8_linear":
            return {**case, "dtype": rng.choice(["bf16", "f16"])}
        return {**case, "out": rng.choice(["bf16", "f16", "f32"])}
    return {"op": op, "tensors": _log_int(rng, 1, 60), "largest": _log_int(rng, 64, 1 << 23),
            "shapes": rng.randrange(1 << 20), "dtype": rng.choice(["bf16", "f32", "mixed"]),
            "ratio": rng.choice([0.1, 0.5, 4.0])}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, d, dtype):
    """Normal values whose columns have unlike magnitudes and means, as hidden states have."""
    x = (_normal(g, rows, d) + 0.5 * _normal(g, d)) * torch.exp(0.7 * _normal(g, d))
    return x.clamp(-400, 400).to(TYPES[dtype]) if dtype == "e4m3" else x.to(TYPES[dtype])


def _blocks(n):
    return (n + 127) // 128


def _choices(g, case):
    """(tokens, top) int64: each token's most likely experts, some of them dropped; skew is the experts' spread."""
    score = _normal(g, case["tokens"], case["experts"]) + case["skew"] * _normal(g, case["experts"])
    expert = torch.topk(score, case["top"], 1).indices
    if case["dropped"]:
        out = torch.rand(case["tokens"], case["top"], generator=g, device="cuda") < case["dropped"]
        expert = torch.where(out, torch.full_like(expert, -1), expert)
    return expert


def _clip_sizes(case):
    """(elements, type) of each tensor: sizes spread over their logarithm, and the first one of the largest size."""
    r = random.Random(case["shapes"])
    sizes = [case["largest"]] + [_log_int(r, 1, case["largest"]) for _ in range(case["tensors"] - 1)]
    kinds = ["bf16", "f32"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [(n, r.choice(kinds)) for n in sizes]


GRADIENT = 0.01  # spread of a gradient's elements


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    new = lambda *shape, t: torch.empty(*shape, dtype=TYPES.get(t, t), device="cuda")  # noqa: E731
    s = {"case": case}
    if op in ("dispatch", "combine", "combine_backward"):
        tokens, top, d, dtype = case["tokens"], case["top"], case["d"], case["dtype"]
        n = tokens * top
        expert = _choices(g, case)
        if op == "dispatch":
            s["expert"] = expert
            s["x"] = _activations(g, tokens, d, dtype)
            if dtype == "e4m3":
                s["scale"] = torch.exp(_normal(g, _blocks(d), tokens))
                s["scale_out"] = new(_blocks(d), n, t="f32")
            s["sizes"], s["choice"] = new(case["experts"], t=torch.int32), new(n, t=torch.int32)
            s["row"] = new(tokens, top, t=torch.int32)
            s["rows"] = new(n, d, t=dtype)
        else:
            s["sizes"], s["row"], s["choice"] = _sorted(expert, case["experts"])
            s["weight"] = torch.softmax(_normal(g, tokens, top), 1)
            s["rows"] = _normal(g, n, d).to(TYPES[dtype])
            if op == "combine":
                s["y"] = new(tokens, d, t=dtype)
            else:
                s["dy"] = (0.01 * _normal(g, tokens, d)).to(TYPES[dtype])
                s["drows_in"] = (0.01 * _normal(g, n, d)).to(TYPES[dtype])
                s["drows"], s["dweight"] = new(n, d, t=dtype), new(tokens, top, t="f32")
                s["dx"] = new(tokens, d, t=dtype)
    elif op in ("layer_norm", "layer_norm_backward"):
        rows, d, dtype = case["rows"], case["d"], case["dtype"]
        s["weight"] = (1 + 0.2 * _normal(g, d)).to(TYPES[dtype])
        if op == "layer_norm":
            s["bias"] = (0.2 * _normal(g, d)).to(TYPES[dtype])
            s["x"] = _activations(g, rows, d, dtype)
            s["residual"] = _activations(g, rows, d, dtype) if case["residual"] else None
            s["y"] = new(rows, d, t=dtype)
            s["h"] = new(rows, d, t=dtype) if case["residual"] else None
        else:
            s["h"] = _activations(g, rows, d, dtype)
            h = s["h"].float()
            s["mean"] = h.mean(1)
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = (0.01 * _normal(g, rows, d)).to(TYPES[dtype])
            s["dh"] = (0.01 * _normal(g, rows, d)).to(TYPES[dtype])
            s["dx"] = new(rows, d, t=dtype)
            s["dweight"], s["dbias"] = new(d, t="f32"), new(d, t="f32")
    elif op in ("int8_linear", "gemm_int8"):
        m, n, k = case["m"], case["n"], case["k"]
        s["b"], s["sb"] = _quantize(_normal(g, n, k) / math.sqrt(k))
        if op == "int8_linear":
            s["x"] = _activations(g, m, k, case["dtype"])
            s["a"], s["sa"] = new(m, k, t=torch.int8), new(m, t="f32")
            s["c"] = new(m, n, t=case["dtype"])
        else:
            s["a"], s["sa"] = _quantize(_activations(g, m, k, "f32"))
            s["c"] = new(m, n, t=case["out"])
    else:
        sizes = _clip_sizes(case)
        s["grads"] = [(GRADIENT * _normal(g, n)).to(TYPES[t]) for n, t in sizes]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["max_norm"] = case["ratio"] * GRADIENT * math.sqrt(sum(n for n, _ in sizes))
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _sorted(expert, experts):
    """(sizes, row, choice) of the stable order of the choices by expert."""
    flat = expert.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    sizes = torch.zeros(experts + 1, dtype=torch.int32, device=key.device)
    sizes.scatter_add_(0, key, torch.ones_like(key, dtype=torch.int32))
    row = torch.where(key < experts, place, ~place).to(torch.int32)
    choice = torch.where(key[order] < experts, order, ~order).to(torch.int32)
    return sizes[:experts].clone(), row.view(expert.shape), choice


def _quantize(x):
    """(int8 values, scales): scale = the row's largest magnitude / 127."""
    x = x.float()
    scale = x.abs().amax(1).clamp(min=SMALLEST_AMAX) / 127
    return torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _of_choices(rows, row):
    """(tokens, top, d) float32: the rows of each token's choices, zero where dropped."""
    return torch.where((row >= 0)[..., None], rows.float()[row.clamp(min=0)], 0)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        sizes, row, choice = _sorted(s["expert"], case["experts"])
        token = torch.where(choice < 0, ~choice, choice) // case["top"]
        routed = choice >= 0
        if case["dtype"] == "e4m3":  # torch indexes and masks these as bytes
            rows = torch.where(routed[:, None], s["x"].view(torch.uint8)[token], 0).view(TYPES["e4m3"])
            return sizes, row, choice, rows, torch.where(routed, s["scale"][:, token], 0)
        return sizes, row, choice, torch.where(routed[:, None], s["x"][token], 0)
    if op == "combine":
        y = (_of_choices(s["rows"], s["row"]) * s["weight"][..., None]).sum(1)
        return y.to(TYPES[case["dtype"]])
    if op == "combine_backward":
        row, dy = s["row"], s["dy"].float()
        dweight = (_of_choices(s["rows"], row) * dy[:, None, :]).sum(2)
        token = torch.where(s["choice"] < 0, ~s["choice"], s["choice"]).long()
        drows = dy[token // case["top"]] * s["weight"].view(-1)[token][:, None]
        drows = torch.where((s["choice"] >= 0)[:, None], drows, 0)
        dx = _of_choices(s["drows_in"], row).sum(1)
        return drows.to(TYPES[case["dtype"]]), dweight, dx.to(TYPES[case["dtype"]])
    if op == "layer_norm":
        x = s["x"].float()
        h = x + s["residual"].float() if case["residual"] else x
        c = h - h.mean(1, keepdim=True)
        y = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["weight"].float() + s["bias"].float()
        return y.to(TYPES[case["dtype"]]), h.to(TYPES[case["dtype"]]) if case["residual"] else None
    if op == "layer_norm_backward":
        xhat = (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        inner = g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)
        dx = s["dh"].float() + s["rstd"][:, None] * inner
        return dx.to(TYPES[case["dtype"]]), (dy * xhat).sum(0), dy.sum(0)
    if op == "clip":
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
        factor = (s["max_norm"] / (norm + NORM_EPS)).clamp(max=1)
        return norm, [(t.float() * factor).to(t.dtype) for t in s["grads"]]
    a, sa = _quantize(s["x"]) if op == "int8_linear" else (s["a"], s["sa"])
    c = (a.float() @ s["b"].float().t()) * sa[:, None] * s["sb"]
    return c.to(s["c"].dtype)


# ---- the library's calls -----------------------------------------------------------------------------------------

def _library(s):
    import tile_size_selection_amd as tss
    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        order = tss.sort_by_expert(s["expert"], case["experts"], sizes=s["sizes"], row=s["row"], choice=s["choice"])
        if case["dtype"] == "e4m3":
            rows, scale = tss.gather_rows(s["x"], order, s["scale"], out=s["rows"], scale_out=s["scale_out"])
            return order.sizes, order.row, order.choice, rows, scale
        return order.sizes, order.row, order.choice, tss.gather_rows(s["x"], order, out=s["rows"])
    if op in ("combine", "combine_backward"):
        order = tss.ExpertOrder(s["sizes"], s["row"], s["choice"])
        if op == "combine":
            return tss.combine_rows(s["rows"], order, s["weight"], out=s["y"])
        drows, dweight = tss.combine_rows_backward(s["dy"], s["rows"], order, s["weight"], drows=s["drows"],
                                                   dweight=s["dweight"])
        return drows, dweight, tss.gather_rows_backward(s["drows_in"], order, out=s["dx"])
    if op == "layer_norm":
        r = tss.layer_norm(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS, out=s["y"], residual_out=s["h"])
        return r.y, r.h
    if op == "layer_norm_backward":
        return tss.layer_norm_backward(s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], s["dh"], dx=s["dx"],
                                       dweight=s["dweight"], dbias=s["dbias"])
    if op == "clip":
        return tss.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]), s["out"]
    if op == "int8_linear":
        a, sa = tss.quantize_int8(s["x"], out=s["a"], scale=s["sa"])
        return tss.gemm_int8(a, s["b"], sa, s["sb"], out_dtype=case["dtype"], out=s["c"])
    return tss.gemm_int8(s["a"], s["b"], s["sa"], s["sb"], out_dtype=case["out"], out=s["c"])


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_backward"):
        tokens, top, d, size = case["tokens"], case["top"], case["d"], SIZE[case["dtype"]]
        n = tokens * top
        kept = n * (1 - case["dropped"])  # rows that are read
        if op == "dispatch":
            scales = 4 * _blocks(d) * (tokens + n) if case["dtype"] == "e4m3" else 0
            return {"bytes": int((tokens + n) * d * size + scales + 8 * n + 8 * n + 4 * case["experts"]), "flops": n}
        if op == "combine":
            return {"bytes": int((kept + tokens) * d * size + 8 * n), "flops": int(2 * kept * d)}
        # rows, dy, the rows' gradients to be summed; the rows' gradients, dx; row and weight, dweight
        return {"bytes": int((2 * kept + n + 2 * tokens) * d * size + 12 * n), "flops": int(4 * kept * d)}
    if op in ("layer_norm", "layer_norm_backward"):
        d, size = case["d"], SIZE[case["dtype"]]
        n = case["rows"] * d
        if op == "layer_norm":
            return {"bytes": n * size * (4 if case["residual"] else 2) + 2 * d * size, "flops": 8 * n}
        return {"bytes": 4 * n * size + 8 * case["rows"] + d * size + 8 * d, "flops": 14 * n}
    if op == "clip":
        sizes = _clip_sizes(case)
        return {"bytes": sum(2 * n * SIZE[t] for n, t in sizes) + 4, "flops": sum(3 * n for n, _ in sizes)}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "int8_linear":
        return {"bytes": m * k * SIZE[case["dtype"]] + n * k + 4 * n + m * n * SIZE[case["dtype"]], "flops": 2 * m * n * k}
    return {"bytes": m * k + n * k + 4 * (m + n) + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}


# ---- the definition in 64 bits -----------------------------------------------------------------------------------

def _exact_order(expert, experts):
    """(sizes, row, choice), expert by expert."""
    flat = expert.flatten()
    members = [(flat == e).nonzero()[:, 0] for e in range(experts)]
    members.append(((flat < 0) | (flat >= experts)).nonzero()[:, 0])
    sizes = torch.tensor([len(m) for m in members[:-1]], dtype=torch.int32, device=flat.device)
    choice = torch.cat(members)
    row = torch.empty_like(choice)
    row[choice] = torch.arange(len(choice), device=flat.device)
    routed = int(sizes.sum())
    row = torch.where(row >= routed, -row - 1, row)
    choice = torch.cat([choice[:routed], -choice[routed:] - 1])
    return sizes, row.view(expert.shape).int(), choice.int()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        sizes, row, choice = _exact_order(s["expert"], case["experts"])
        x = s["x"].double()
        rows = torch.zeros(len(choice), case["d"], dtype=torch.float64, device="cuda")
        scale = torch.zeros(_blocks(case["d"]), len(choice), dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            t = (row[:, j] >= 0).nonzero()[:, 0]
            r = row[t, j].long()
            rows[r] = x[t]
            if case["dtype"] == "e4m3":
                scale[:, r] = s["scale"].double()[:, t]
        return (sizes, row, choice, rows) + ((scale,) if case["dtype"] == "e4m3" else ())
    if op in ("combine", "combine_backward"):
        row, w, tokens = s["row"], s["weight"].double(), case["tokens"]
        y = torch.zeros(tokens, case["d"], dtype=torch.float64, device="cuda")
        if op == "combine":
            for j in range(case["top"]):
                t = (row[:, j] >= 0).nonzero()[:, 0]
                y[t] += w[t, j, None] * s["rows"][row[t, j].long()].double()
            return y
        drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        dweight = torch.zeros_like(w)
        for j in range(case["top"]):
            t = (row[:, j] >= 0).nonzero()[:, 0]
            r, dy = row[t, j].long(), s["dy"][t].double()
            drows[r] = w[t, j, None] * dy
            dweight[t, j] = torch.linalg.vecdot(dy, s["rows"][r].double())
            y[t] += s["drows_in"][r].double()
        return drows, dweight, y
    if op == "layer_norm":
        h = s["x"].double()
        if case["residual"]:
            h = h + s["residual"].double()
        var, mean = torch.var_mean(h, 1, correction=0, keepdim=True)
        y = torch.addcmul(s["bias"].double(), (h - mean) / torch.sqrt(var + EPS), s["weight"].double())
        return y, h if case["residual"] else None
    if op == "layer_norm_backward":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        c = h - s["mean"].double()[:, None]
        g = dy * s["weight"].double()
        d = case["d"]
        inner = torch.linalg.vecdot(g, c)[:, None]
        dx = r * g - r * (g.sum(1, keepdim=True) / d) - c * (r ** 3 * inner / d) + s["dh"].double()
        return dx, torch.linalg.vecdot(dy.t(), (c * r).t()), torch.linalg.vecdot(dy.t(), torch.ones_like(dy).t())
    if op == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]))
        factor = min(1.0, s["max_norm"] / (float(norm) + NORM_EPS))
        return norm, [t.double() * factor for t in s["grads"]]
    if op == "int8_linear":
        x = s["x"].double()
        sa = torch.linalg.vector_norm(x, math.inf, dim=1).clamp(min=SMALLEST_AMAX) / 127
        a = torch.round(x / sa[:, None])
    else:
        a, sa = s["a"].double(), s["sa"].double()
    return (a @ s["b"].double().t()).mul_(sa[:, None]).mul_(s["sb"].double())
