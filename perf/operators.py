"""The operators of a routed FFN, as a user calls them, with their plain forms.

A layer whose FFN is split into experts sends each token to the `top_k` experts
with the largest logits, runs the rows of each expert through that expert's own
matrices and adds a token's rows up again with the router's weights:

    route     top_k experts of every token, their softmax weights, and the plan
              that lists the rows expert by expert
    grouped   out[r] = a[row_index[r]] W_g^T for the rows r of group g, ragged;
              gated: (a W_up^T) * SiLU(a W_gate^T)
    fp8       the same product of e4m3 values with one fp32 scale for each 128
              inputs of a row and for each 128 x 128 block of the weights; dense
              (one group) or by expert
    quantize  rows to e4m3 with a scale for each 128 values
    combine   y[t] = sum over slots s of weight[t, s] h[row_of[t, s]]

`own` false: the plain forms, in fp32 torch.  `own` true: the library's calls.
"""
import math

import torch
import torch.nn.functional as F

own = False

def _library():
    from free_ffn_activation_amd import prox
    return prox


FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": FP8}
SIZE = {"f32": 4, "bf16": 2, "fp8": 1}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token: latency only
        {"name": "route_one", "op": "route", "tokens": 1, "experts": 64, "top_k": 8, "dtype": "f32",
         "renorm": True, "masked": 0.0},
        # a prompt with some padded positions (all logits -inf), bf16 logits as a bf16 layer makes them (many ties)
        {"name": "route_prompt", "op": "route", "tokens": 8191, "experts": 128, "top_k": 8, "dtype": "bf16",
         "renorm": True, "masked": 0.05},
        # one decoded token through its 8 experts' up/gate matrices: a weight stream
        {"name": "upgate_one", "op": "grouped", "tokens": 1, "experts": 64, "top_k": 8, "k": 2048, "n": 1024,
         "gated": True, "gather": True, "dtype": "bf16", "out": "bf16", "masked": 0.0},
        # a decode batch of 61 sequences, down projection: every expert has a few rows
        {"name": "down_batch", "op": "grouped", "tokens": 61, "experts": 64, "top_k": 8, "k": 1024, "n": 2048,
         "gated": False, "gather": False, "dtype": "bf16", "out": "bf16", "masked": 0.0},
        # a prompt of 8192 tokens: about 1024 ragged rows for each expert; the largest
        {"name": "upgate_prompt", "op": "grouped", "tokens": 8192, "experts": 64, "top_k": 8, "k": 2048, "n": 1024,
         "gated": True, "gather": True, "dtype": "bf16", "out": "bf16", "masked": 0.0},
        # an fp32 layer of the framework's smallest configuration (256 x 768) with experts
        {"name": "down_f32", "op": "grouped", "tokens": 517, "experts": 16, "top_k": 2, "k": 768, "n": 256,
         "gated": False, "gather": False, "dtype": "f32", "out": "f32", "masked": 0.0},
        # the Qwen3-8B-shaped down projection in fp8 for seven decoded tokens: a weight stream
        {"name": "fp8_decode", "op": "grouped", "tokens": 7, "experts": 1, "top_k": 1, "k": 12288, "n": 4096,
         "gated": False, "gather": False, "dtype": "fp8", "out": "bf16", "masked": 0.0},
        # one Qwen3-8B-shaped projection in fp8 over a prompt
        {"name": "fp8_prompt", "op": "grouped", "tokens": 4000, "experts": 1, "top_k": 1, "k": 4096, "n": 12288,
         "gated": False, "gather": False, "dtype": "fp8", "out": "bf16", "masked": 0.0},
        # the activations of seven decoded tokens, and of a prompt, to fp8
        {"name": "quantize_one", "op": "quantize", "rows": 7, "k": 12288, "dtype": "bf16", "block_rows": 1},
        {"name": "quantize_prompt", "op": "quantize", "rows": 8192, "k": 4096, "dtype": "bf16", "block_rows": 1},
        # one token's eight expert rows added up, and a prompt's
        {"name": "combine_one", "op": "combine", "tokens": 1, "top_k": 8, "k": 2048, "dtype": "bf16", "out": "f32",
         "masked": 0.0},
        {"name": "combine_prompt", "op": "combine", "tokens": 8192, "top_k": 8, "k": 2048, "dtype": "bf16",
         "out": "bf16", "masked": 0.02},
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "grouped", "fp8", "fp8", "quantize", "combine"])
    masked = rng.choice([0.0, 0.0, 0.1])
    if op == "route":
        e = _span(rng, 4, 256)
        return {"op": op, "tokens": _span(rng, 1, 8192), "experts": e, "top_k": rng.randint(1, min(8, e)),
                "dtype": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.7, "masked": masked}
    if op == "quantize":
        return {"op": op, "rows": _span(rng, 1, 8192), "k": 16 * _span(rng, 8, 256),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "block_rows": rng.choice([1, 1, 1, 128])}
    if op == "combine":
        return {"op": op, "tokens": _span(rng, 1, 8192), "top_k": rng.randint(1, 8), "k": 8 * _span(rng, 16, 256),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"]), "masked": masked}
    dtype = "fp8" if op == "fp8" else rng.choice(["bf16", "bf16", "bf16", "f32"])
    e = rng.choice([1, _span(rng, 2, 128)])
    gated = rng.random() < 0.5
    case = {"op": "grouped", "tokens": _span(rng, 1, 8192), "experts": e, "top_k": rng.randint(1, min(8, e)),
            "k": 16 * _span(rng, 16, 256), "n": _span(rng, 128, 4096), "gated": gated,
            "gather": rng.random() < 0.5, "dtype": dtype, "out": "f32" if dtype == "f32" else "bf16",
            "masked": masked if e > 1 else 0.0}
    most = work(listed()[4])
    if dtype == "f32":  # fp32 products are for small layers
        most = {"bytes": most["bytes"] / 8, "flops": most["flops"] / 32}
    while work(case)["flops"] > most["flops"] or work(case)["bytes"] > most["bytes"]:
        big = max(("tokens", "n", "k"), key=lambda v: case[v])
        case[big] = max(16, case[big] // 32 * 16) if big == "k" else max(1, case[big] * 2 // 3)
    return case


def work(case):
    op, t = case["op"], case.get("tokens")
    if op == "route":
        rows = t * case["top_k"]
        # logits in; ids, weights, row_token, row_of out
        return {"bytes": t * case["experts"] * SIZE[case["dtype"]] + rows * 16 + 4 * (case["experts"] + 1),
                "flops": t * case["experts"] + 4 * rows}
    if op == "quantize":
        n = case["rows"] * case["k"]
        return {"bytes": n * SIZE[case["dtype"]] + n + 4 * n / (128 * case["block_rows"]), "flops": 2 * n}
    if op == "combine":
        n = t * case["k"]
        return {"bytes": n * case["top_k"] * SIZE[case["dtype"]] + n * SIZE[case["out"]] + 8 * t * case["top_k"],
                "flops": 2 * n * case["top_k"]}
    e, rows, n, k = case["experts"], t * case["top_k"], case["n"], case["k"]
    mats = 2 if case["gated"] else 1
    # a token's experts differ, so one expert is without rows with (1 - top_k / experts) ^ tokens
    active = e * (1.0 - (1.0 - case["top_k"] / e) ** t)
    a_rows = t if case["gather"] else rows
    size = SIZE[case["dtype"]]
    scales = (a_rows * k / 128 + active * mats * n * k / 16384) * 4 if case["dtype"] == "fp8" else 0
    return {"bytes": active * mats * n * k * size + a_rows * k * size + rows * n * SIZE[case["out"]] + scales,
            "flops": 2 * mats * rows * n * k}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(g, rows, k):
    """Laplace(0, 1) activations, one coordinate in a thousand 30 times as large (the framework's own tokens)."""
    u = torch.rand(rows, k, device="cuda", generator=g) - 0.5
    x = -torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))
    pos = torch.randperm(k, device="cuda", generator=g)[:max(1, k // 1000)]
    x[:, pos] *= 30.0
    return x


def _logits(g, case):
    t, e = case["tokens"], case["experts"]
    bias = 0.5 * torch.randn(e, device="cuda", generator=g)  # experts are not equally liked
    z = torch.randn(t, e, device="cuda", generator=g) + bias
    pad = torch.rand(t, 1, device="cuda", generator=g) < case["masked"]
    return torch.where(pad, torch.full_like(z, -math.inf), z)


def _blocks(x, rows):
    """e4m3 codes and scales of [..., r, k], one scale for each rows x 128 block (largest magnitude / 448)."""
    *lead, r, k = x.shape
    p = F.pad(x, (0, -k % 128, 0, -r % rows))
    b = p.reshape(*lead, p.shape[-2] // rows, rows, p.shape[-1] // 128, 128)
    most = b.abs().amax(dim=(-3, -1))
    scale = most / torch.full_like(most, FP8_MAX)  # a division: by a plain number torch multiplies with its inverse
    wide = scale[..., :, None, :, None]
    q = torch.where(wide > 0, b / wide, torch.zeros_like(b)).reshape(p.shape)[..., :r, :k]
    return q.to(FP8).contiguous(), scale.contiguous()


def _widen(scale, rows, r, k):
    """Block scales [..., r / rows, k / 128] as one value for each of the r x k elements."""
    s = scale.repeat_interleave(128, dim=-1)[..., :k]
    return s.repeat_interleave(rows, dim=-2)[..., :r, :] if rows > 1 else s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    new = dict(device="cuda")
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        i32 = dict(dtype=torch.int32, **new)
        s = {"case": case, "logits": _logits(g, case).to(TYPES[case["dtype"]]), "ids": torch.empty(t, k, **i32),
             "weight": torch.empty(t, k, **new), "offsets": torch.empty(e + 1, **i32),
             "row_token": torch.empty(t * k, **i32), "row_of": torch.empty(t, k, **i32)}
        if own:  # the call's workspace
            s["ws"] = torch.empty(_library().prox_expert_route_workspace_size(t, e, k), dtype=torch.uint8, **new)
        return s
    if op == "quantize":
        x = _tokens(g, case["rows"], case["k"]).to(TYPES[case["dtype"]])
        r, kb = -(-case["rows"] // case["block_rows"]), -(-case["k"] // 128)
        return {"case": case, "x": x, "q": torch.empty(x.shape, dtype=FP8, **new), "scale": torch.empty(r, kb, **new)}
    if op == "combine":
        t, k = case["tokens"], case["top_k"]
        order = torch.randperm(t * k, device="cuda", generator=g).reshape(t, k)
        gone = torch.rand(t, 1, device="cuda", generator=g) < case["masked"]
        weight = torch.softmax(torch.randn(t, k, device="cuda", generator=g), 1)
        return {"case": case, "h": torch.randn(t * k, case["k"], device="cuda", generator=g).to(TYPES[case["dtype"]]),
                "row_of": torch.where(gone, torch.full_like(order, -1), order).int(),
                "weight": torch.where(gone, torch.zeros_like(weight), weight),
                "y": torch.empty(t, case["k"], dtype=TYPES[case["out"]], **new)}
    t, e, kk, n, k = case["tokens"], case["experts"], case["top_k"], case["n"], case["k"]
    dt = TYPES[case["dtype"]]
    # the plan that the router gives: rows by expert, tokens ascending within one
    z = _logits(g, case)
    valid = (z > -math.inf).any(1, keepdim=True).expand(t, kk)
    ids = torch.where(valid, torch.topk(z, kk, dim=1).indices, torch.full((t, kk), e, **new)).reshape(-1)
    order = torch.argsort(ids, stable=True)
    sizes = torch.bincount(ids, minlength=e + 1)[:e]
    offsets = torch.zeros(e + 1, dtype=torch.int32, **new)
    offsets[1:] = torch.cumsum(sizes, 0)
    token = (order // kk).int()
    used = torch.arange(t * kk, **new) < offsets[-1]
    x = _tokens(g, t, k)
    w = torch.randn(2 if case["gated"] else 1, e, n, k, device="cuda", generator=g) * 0.02
    s = {"case": case, "offsets": offsets, "row_index": torch.where(used, token, torch.full_like(token, -1))}
    rows = x if case["gather"] else x[token.long()]
    if dt is FP8:
        s["a"], s["a_scale"] = _blocks(rows.to(torch.bfloat16).float(), 1)
        for i, name in enumerate(("w", "w_gate")[:len(w)]):
            s[name], s[name + "_scale"] = _blocks(w[i].to(torch.bfloat16).float(), 128)
    else:
        s["a"] = rows.to(dt)
        for i, name in enumerate(("w", "w_gate")[:len(w)]):
            s[name] = w[i].to(dt)
    # rows behind the last group are left as they were
    s["out"] = torch.zeros(t * kk, n, dtype=TYPES[case["out"]], **new)
    # what a padded batched product has to know of the groups: those with rows, and each row's place in it
    live = torch.nonzero(sizes).reshape(-1)
    s["live"], s["most"] = live, int(sizes.max())
    group = torch.repeat_interleave(torch.arange(live.numel(), **new), sizes[live])
    s["place"] = group * s["most"] + torch.arange(group.numel(), **new) - offsets[:-1][live].long()[group]
    if own:  # the layer's handle
        s["experts"] = _library().ProxExperts(s["w"], s.get("w_gate"), scale=s.get("w_scale"),
                                              gate_scale=s.get("w_gate_scale"))
    return s


# ------------------------------------------------------------------- the runs
def run(s):
    op = s["case"]["op"]
    return {"route": _route, "quantize": _quantize, "combine": _combine, "grouped": _grouped}[op](s)


def _route(s):
    case = s["case"]
    if own:
        _library().prox_expert_route(s["logits"], s["ids"], s["weight"], s["offsets"], s["row_token"], s["row_of"], s["ws"],
                            renormalize=case["renorm"])
        return [s[v] for v in ("ids", "weight", "offsets", "row_token", "row_of")]
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    z = s["logits"].float()
    top, idx = torch.sort(z, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    valid = top > -math.inf
    ids = torch.where(valid, idx, torch.full_like(idx, -1))
    base = torch.where(valid[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    p = torch.exp(top - base)
    total = p.sum(1, keepdim=True) if case["renorm"] else torch.exp(z - base).sum(1, keepdim=True)
    weight = torch.where(valid, p / total, torch.zeros_like(p))
    key = torch.where(valid, idx, torch.full_like(idx, e)).reshape(-1)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(e + 1, dtype=torch.int64, device=z.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = F.pad(torch.cumsum(count[:e], 0), (1, 0))
    at = torch.arange(t * k, device=z.device)
    row_token = torch.where(at < offsets[-1], order // k, torch.full_like(order, -1))
    row_of = torch.empty_like(at).scatter_(0, order, at).reshape(t, k)
    row_of = torch.where(valid, row_of, torch.full_like(row_of, -1))
    return [ids.int(), weight, offsets.int(), row_token.int(), row_of.int()]


def _quantize(s):
    rows = s["case"]["block_rows"]
    if own:
        _library().prox_fp8_quantize(s["x"], s["q"], s["scale"], block_rows=rows)
        return [s["q"], s["scale"]]
    return list(_blocks(s["x"].float(), rows))


def _combine(s):
    if own:
        _library().prox_expert_combine(s["h"], s["row_of"], s["weight"], s["y"])
        return s["y"]
    kept = s["row_of"] >= 0
    h = s["h"][s["row_of"].clamp(min=0).long()].float()
    y = (h * torch.where(kept, s["weight"], torch.zeros_like(s["weight"]))[:, :, None]).sum(1)
    return y.to(TYPES[s["case"]["out"]])


def _grouped(s):
    case = s["case"]
    if own:
        _library().prox_grouped_matmul(s["experts"], s["a"], s["out"], offsets=s["offsets"],
                              row_index=s["row_index"] if case["gather"] else None, a_scale=s.get("a_scale"))
        return s["out"]
    n, k, used = case["n"], case["k"], s["place"].numel()
    a = s["a"].float()
    if "a_scale" in s:
        a = a * _widen(s["a_scale"], 1, a.shape[0], k)
    a = a[s["row_index"][:used].long()] if case["gather"] else a[:used]
    padded = torch.zeros(s["live"].numel() * s["most"], k, device=a.device)
    padded[s["place"]] = a
    padded = padded.reshape(-1, s["most"], k)
    outs = [torch.bmm(padded, _weights(s, name).transpose(1, 2)) for name in ("w", "w_gate") if name in s]
    h = outs[0] * (outs[1] * torch.sigmoid(outs[1])) if case["gated"] else outs[0]
    out = torch.zeros_like(s["out"])
    out[:used] = h.reshape(-1, n)[s["place"]].to(out.dtype)
    return out


def _weights(s, name):
    w = s[name][s["live"]].float()
    if name + "_scale" in s:
        w = w * _widen(s[name + "_scale"][s["live"]], 128, w.shape[1], w.shape[2])
    return w


# ---------------------------------------------------- the definitions in fp64
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits on the same inputs."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        z = s["logits"].double().cpu()
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # descending logit, ascending expert: two stable sorts would do; ranks by counting say it directly
        beats = torch.zeros(t, e, dtype=torch.int64)
        for j in range(e):
            more = z[:, j:j + 1] > z
            same = (z[:, j:j + 1] == z) & (torch.arange(e) > j)
            beats += (more | same) & (z[:, j:j + 1] > -math.inf)
        chosen = (beats < k) & (z > -math.inf)
        shift = torch.nan_to_num(z.amax(1, keepdim=True), neginf=0.0)
        p = torch.exp(z - shift)
        total = torch.where(chosen, p, torch.zeros_like(p)).sum(1) if case["renorm"] else p.sum(1)
        ids = torch.full((t, k), -1, dtype=torch.int32)
        weight = torch.zeros(t, k, dtype=torch.float64)
        tt, ee = torch.nonzero(chosen, as_tuple=True)
        ids[tt, beats[tt, ee]] = ee.int()
        weight[tt, beats[tt, ee]] = p[tt, ee] / total[tt]
        count = chosen.sum(0)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(count, 0)])
        # the row of (token, expert): the expert's first row, and one for each earlier token that has it
        row = offsets[:-1][None] + torch.cumsum(chosen, 0) - 1
        row_of = torch.full((t, k), -1, dtype=torch.int32)
        row_of[tt, beats[tt, ee]] = row[tt, ee].int()
        row_token = torch.full((t * k,), -1, dtype=torch.int32)
        row_token[row[tt, ee]] = tt.int()
        return [ids, weight, offsets.int(), row_token, row_of]
    if op == "quantize":
        rows = case["block_rows"]
        x = s["x"].double()
        r, k = x.shape
        scale = torch.empty(-(-r // rows), -(-k // 128), dtype=torch.float64, device=x.device)
        wide = torch.empty_like(x)
        for c in range(scale.shape[1]):
            most = x[:, 128 * c:128 * c + 128].abs().amax(1)
            if rows > 1:
                most = torch.stack([part.max() for part in torch.split(most, rows)])
            scale[:, c] = (most / FP8_MAX).float()  # the scale is an fp32 value
            wide[:, 128 * c:128 * c + 128] = scale[:, c].repeat_interleave(rows)[:r, None]
        # e4m3: three bits behind the leading one, steps of 2^-9 at the least, ties to even
        v = torch.where(wide > 0, x / wide, torch.zeros_like(x))
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return [torch.round(v / step) * step, scale]
    if op == "combine":
        h, y = s["h"].double(), 0.0
        for j in range(case["top_k"]):
            at = s["row_of"][:, j].long()
            y = y + torch.where(at >= 0, s["weight"][:, j].double(), 0.0)[:, None] * h[at.clamp(min=0)]
        return y
    if work(case)["flops"] > 6e11:
        return None
    bounds = s["offsets"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for g in range(case["experts"]):
        lo, hi = bounds[g], bounds[g + 1]
        if hi == lo:
            continue
        at = s["row_index"][lo:hi].long() if case["gather"] else slice(lo, hi)
        a = s["a"][at].double()
        if "a_scale" in s:
            a *= torch.repeat_interleave(s["a_scale"][at].double(), 128, 1)[:, :a.shape[1]]
        got = []
        for name in ("w", "w_gate")[:2 if case["gated"] else 1]:
            w = s[name][g].double()
            if name + "_scale" in s:
                b = s[name + "_scale"][g].double()
                rows_of = torch.arange(w.shape[0], device="cuda") // 128
                w *= b[rows_of][:, torch.arange(w.shape[1], device="cuda") // 128]
            got.append(a @ w.T)
        out[lo:hi] = got[0] * got[1] / (1.0 + torch.exp(-got[1])) if case["gated"] else got[0]
    return out
