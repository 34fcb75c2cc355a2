"""Timed cases of the operators around a projection: the RMS norm with the
residual's addition (bf16 or E4M3FN rows) and its gradient, the projection
with low-rank adapters of many requests, and the mixture-of-experts SwiGLU
layer for a few tokens.

`run` computes each operator either by the library's kernels (`own`) or in
its plain form: elementary torch operations in 32 bits, rounded at the end.
`exact` computes it in 64 bits, apart from both.
"""
import math

import torch

own = False

EPS = 1e-6
_kept = {}


def listed():
    return [
        # a single token's hidden state between two projections: latency only
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "codes": False, "residual": True},
        # a batch before an FP8 projection: rows leave as codes with factors
        {"name": "norm_codes_batch", "op": "norm", "rows": 1024, "cols": 4096, "codes": True, "residual": True},
        # a long prompt or a training batch, wide rows
        {"name": "norm_long", "op": "norm", "rows": 16384, "cols": 8192, "codes": False, "residual": True},
        # the gradient in a training step, with the residual branch's gradient
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "cols": 4096, "residual": True},
        # the same for a ragged batch, no residual branch
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 1000, "cols": 4100, "residual": False},
        # one request with its adapter
        {"name": "lora_token", "op": "lora", "rows": 1, "n": 12288, "k": 4096, "rank": 16, "adapters": 8,
         "order": "mixed"},
        # a decoding step of sixteen requests, each with an adapter of its own
        {"name": "lora_decode", "op": "lora", "rows": 16, "n": 12288, "k": 4096, "rank": 16, "adapters": 64,
         "order": "mixed"},
        # odd sizes, a larger rank, rows of different requests between each other
        {"name": "lora_ragged", "op": "lora", "rows": 77, "n": 4104, "k": 4100, "rank": 24, "adapters": 16,
         "order": "mixed"},
        # prompts of several requests behind each other
        {"name": "lora_prompts", "op": "lora", "rows": 1024, "n": 12288, "k": 4096, "rank": 16, "adapters": 8,
         "order": "runs"},
        # one token through the expert layer
        {"name": "experts_token", "op": "experts", "tokens": 1, "hidden": 4096, "inner": 1536, "experts": 64,
         "topk": 8, "codes": False, "renormalize": True},
        # a decoding step of sixteen requests
        {"name": "experts_decode", "op": "experts", "tokens": 16, "hidden": 4096, "inner": 1536, "experts": 64,
         "topk": 8, "codes": False, "renormalize": True},
        # a larger batch with weights held as E4M3FN codes
        {"name": "experts_codes", "op": "experts", "tokens": 64, "hidden": 4096, "inner": 1536, "experts": 64,
         "topk": 8, "codes": True, "renormalize": False},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v // step, -(-lo // step)), hi // step) * step


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "lora", "lora", "experts", "experts"])
    step = rng.choice([1, 8, 8, 64])     # odd sizes, whole 16-byte chunks, whole matrix-core steps
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 8192, step)
        rows = _log(rng, 1, min(16384, (16384 * 8192) // (cols * (1 if op == "norm" else 4))))
        case = {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7}
        if op == "norm":
            case["codes"] = rng.random() < 0.5
        return case
    if op == "lora":
        return {"op": op, "rows": _log(rng, 1, 1024), "n": _log(rng, 512, 12288, step),
                "k": _log(rng, 512, 4096, step), "rank": _log(rng, 4, 64, rng.choice([1, 4, 8])),
                "adapters": _log(rng, 1, 64), "order": rng.choice(["mixed", "runs"])}
    experts = _log(rng, 4, 64)
    return {"op": op, "tokens": _log(rng, 1, 64), "hidden": _log(rng, 256, 4096, step),
            "inner": _log(rng, 64, 1536, step), "experts": experts, "topk": rng.randint(1, min(8, experts)),
            "codes": rng.random() < 0.5, "renormalize": rng.random() < 0.5}


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        s["w"] = (1.0 + 0.1 * torch.randn((cols,), generator=g, device="cuda")).bfloat16()
        if case["op"] == "norm":
            s["x"] = _normal(g, (rows, cols))
            s["r"] = _normal(g, (rows, cols), 4.0) if case["residual"] else None
        else:
            s["h"] = _normal(g, (rows, cols), 2.0)
            s["dy"] = _normal(g, (rows, cols), 0.01)
            s["dh"] = _normal(g, (rows, cols), 0.01) if case["residual"] else None
            # what the forward call left for the gradient
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
    elif case["op"] == "lora":
        rows, n, k, rank, adapters = (case[q] for q in ("rows", "n", "k", "rank", "adapters"))
        s["x"] = _normal(g, (rows, k))
        s["w"] = _normal(g, (n, k), k ** -0.5)
        s["a"] = _normal(g, (adapters, rank, k), k ** -0.5)
        s["b"] = _normal(g, (adapters, n, rank), rank ** -0.5)
        s["scale"] = torch.rand((adapters,), generator=g, device="cuda") + 0.5
        # each row's adapter, about one in nine rows without any (-1)
        pick = torch.randint(0, adapters, (rows,), generator=g, device="cuda", dtype=torch.int32)
        if rows > 1:
            pick = torch.where(torch.rand((rows,), generator=g, device="cuda") < 1 / 9, -1, pick).to(torch.int32)
        s["idx"] = pick.sort().values if case["order"] == "runs" else pick
    else:
        t, h, i, e = case["tokens"], case["hidden"], case["inner"], case["experts"]
        s["x"] = _normal(g, (t, h))
        s["logits"] = torch.randn((t, e), generator=g, device="cuda")
        if case["codes"]:
            # E4M3FN codes of normal weights, a factor for each row
            s["wgu"] = _normal(g, (e, 2 * i, h), 100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s["wd"] = _normal(g, (e, h, i), 100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s["sgu"] = (torch.rand((e, 2 * i), generator=g, device="cuda") + 0.5) * (0.01 * h ** -0.5)
            s["sd"] = (torch.rand((e, h), generator=g, device="cuda") + 0.5) * (0.01 * i ** -0.5)
        else:
            s["wgu"] = _normal(g, (e, 2 * i, h), h ** -0.5)
            s["wd"] = _normal(g, (e, h, i), i ** -0.5)
            s["sgu"] = s["sd"] = None
    return s


def _workspace(lib):
    """The process's one workspace, as a program that makes these calls in turn keeps it."""
    if "workspace" not in _kept:
        _kept["workspace"] = lib.Workspace()
    return _kept["workspace"]


def _run_own(s):
    import dense_gemm_05_amd as lib
    case = s["case"]
    if case["op"] == "norm":
        f = lib.rms_norm_e4m3 if case["codes"] else lib.rms_norm
        out = f(s["x"], s["w"], residual=s["r"], eps=EPS)
        if case["codes"]:
            return (out[0].view(torch.float8_e4m3fn),) + tuple(out[1:])
        return out
    if case["op"] == "norm_grad":
        return lib.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dH=s["dh"], workspace=_workspace(lib))
    if case["op"] == "lora":
        return lib.gemm_bf16_nt_lora(s["x"], s["w"], s["a"], s["b"], s["idx"], scale=s["scale"],
                                     workspace=_workspace(lib))
    return lib.moe_swiglu(s["x"], s["logits"], case["topk"], s["wgu"], s["wd"], scale_gu=s["sgu"],
                          scale_d=s["sd"], renormalize=case["renormalize"], workspace=_workspace(lib))


def _plain_norm(s):
    x = s["x"].float()
    if s["r"] is not None:
        h = (x + s["r"].float()).bfloat16()     # the residual stream, stored in bf16
        x = h.float()
    y = (x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w"].float()).bfloat16()
    more = () if s["r"] is None else (h,)
    if not s["case"]["codes"]:
        return (y,) + more if more else y
    # the codes of the bf16 rows, a factor for each row
    y = y.float()
    amax = y.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, y * 448.0 / amax, y * 0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (q, amax[:, 0] / 448.0) + more


def _plain_norm_grad(s):
    dy, h, w, rstd = s["dy"].float(), s["h"].float(), s["w"].float(), s["rstd"][:, None]
    xh, g = h * rstd, dy * w
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.bfloat16(), (dy * xh).sum(0)


def _plain_lora(s):
    x, idx = s["x"].float(), s["idx"].long()
    y = x @ s["w"].float().t()
    adapters, rank = s["a"].shape[:2]
    # every adapter's low-rank values, each row keeping those of its own
    # (none: zeros), then one product with all adapters' second halves
    v = (x @ s["a"].float().reshape(adapters * rank, -1).t()).reshape(-1, adapters, rank)
    mine = idx[:, None] == torch.arange(adapters, device=idx.device)
    v = torch.where(mine[:, :, None], v * s["scale"][None, :, None], 0.0).reshape(-1, adapters * rank)
    y = y + v @ s["b"].float().permute(0, 2, 1).reshape(adapters * rank, -1)
    return y.bfloat16()


def _plain_experts(s):
    case, x = s["case"], s["x"].float()
    t, h = x.shape
    k, i, e = case["topk"], case["inner"], case["experts"]
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    over = top if case["renormalize"] else order.values
    p = torch.exp(over - order.values[:, :1])
    gates = p[:, :k] / p.sum(1, keepdim=True)
    if t * k <= e:
        # few pairs of token and expert: the weights of each pair
        wgu, wd = s["wgu"][ids.reshape(-1)].float(), s["wd"][ids.reshape(-1)].float()
        if s["sgu"] is not None:
            wgu, wd = wgu * s["sgu"][ids.reshape(-1)][..., None], wd * s["sd"][ids.reshape(-1)][..., None]
        z = torch.bmm(wgu, x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        z = z[:, :i] * torch.sigmoid(z[:, :i]) * z[:, i:]
        y = torch.bmm(wd, z[:, :, None])[..., 0].reshape(t, k, h)
        y = (y * gates[:, :, None]).sum(1)
    else:
        # every expert on every token, weighted by its gate (0 where not chosen)
        wgu, wd = s["wgu"].float(), s["wd"].float()
        if s["sgu"] is not None:
            wgu, wd = wgu * s["sgu"][..., None], wd * s["sd"][..., None]
        z = torch.matmul(wgu.reshape(e * 2 * i, h), x.t()).reshape(e, 2 * i, t)
        z = z[:, :i] * torch.sigmoid(z[:, :i]) * z[:, i:]
        g = torch.zeros((t, e), device=x.device).scatter_(1, ids, gates)
        y = torch.bmm(wd, z * g.t()[:, None, :]).sum(0).t()
    return y.bfloat16(), ids.to(torch.int32), gates


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_grad":
        return _plain_norm_grad(state)
    if op == "lora":
        return _plain_lora(state)
    return _plain_experts(state)


def _occupied(balls, boxes):
    """How many of `boxes` adapters or experts occur, in the mean over inputs."""
    return boxes * (1.0 - (1.0 - 1.0 / boxes) ** balls)


def work(case):
    if case["op"] == "norm":
        rows, cols, r = case["rows"], case["cols"], 4 if case["residual"] else 0
        return {"bytes": rows * cols * (2 + r + (1 if case["codes"] else 2)) + 2 * cols, "flops": 6 * rows * cols}
    if case["op"] == "norm_grad":
        rows, cols, r = case["rows"], case["cols"], 2 if case["residual"] else 0
        return {"bytes": rows * cols * (6 + r) + 6 * cols + 4 * rows, "flops": 10 * rows * cols}
    if case["op"] == "lora":
        m, n, k, rank = case["rows"], case["n"], case["k"], case["rank"]
        used = _occupied(m, case["adapters"])
        return {"bytes": 2 * (m * k + n * k + m * n + used * rank * (n + k)), "flops": 2 * m * (n * k + rank * (n + k))}
    t, h, i, k = case["tokens"], case["hidden"], case["inner"], case["topk"]
    used = case["experts"] * (1.0 - (1.0 - k / case["experts"]) ** t)
    return {"bytes": used * 3 * i * h * (1 if case["codes"] else 2) + 4 * t * h + 4 * t * case["experts"],
            "flops": 6 * t * k * h * i}


def _nearest_e4m3(q):
    """The E4M3FN value nearest to each |q| <= 448, ties to the even mantissa."""
    exponent = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(q / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        more = ()
        if s["r"] is not None:
            h = h.add(s["r"].double()).bfloat16().double()
            more = (h,)
        y = h / torch.sqrt(torch.mean(h ** 2, dim=1, keepdim=True) + EPS) * s["w"].double()
        if not case["codes"]:
            return (y,) + more if more else y
        y = y.bfloat16().double()
        amax = y.abs().max(dim=1, keepdim=True).values
        return (_nearest_e4m3(448.0 * y / amax.clamp(min=1e-300)), amax[:, 0] / 448.0) + more
    if case["op"] == "norm_grad":
        h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
        rstd = s["rstd"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = rstd * dy * w - h * dot * rstd ** 3 / case["cols"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return dx, torch.mv((dy * h).t(), s["rstd"].double())
    if case["op"] == "lora":
        x = s["x"].double()
        y = torch.mm(x, s["w"].double().t())
        for a in range(case["adapters"]):
            rows = torch.nonzero(s["idx"] == a)[:, 0]
            if rows.numel():
                v = torch.mm(x[rows], s["a"][a].double().t())
                y[rows] += float(s["scale"][a]) * torch.mm(v, s["b"][a].double().t())
        return y
    x, logits, k, i = s["x"].double(), s["logits"].double(), case["topk"], case["inner"]
    # the k largest, ties to the lowest index: numpy's stable sort of the negated logits
    ids = torch.from_numpy((-logits.cpu().numpy()).argsort(axis=1, kind="stable")[:, :k].copy()).to(x.device)
    top = logits.gather(1, ids)
    gates = torch.softmax(top, 1) if case["renormalize"] else torch.softmax(logits, 1).gather(1, ids)
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        wgu, wd = s["wgu"][e].double(), s["wd"][e].double()
        if case["codes"]:
            wgu, wd = wgu * s["sgu"][e].double()[:, None], wd * s["sd"][e].double()[:, None]
        z = torch.mm(x[t], wgu.t())
        z = torch.nn.functional.silu(z[:, :i]) * z[:, i:]
        y[t] += gates[t, slot][:, None] * torch.mm(z, wd.t())
    return y, ids.to(torch.int32), gates
