"""Timed cases of what a training step computes at both ends of the
projections: the loss over a large vocabulary behind the last projection, from
labels or from a teacher's top logits, alone and with its gradient, and the
experts' products with ragged numbers of rows, forward and both gradients.

`run` computes each operator either by the library's kernels (`own`) or in
its plain form: elementary torch operations in 32 bits, rounded at the end.
`exact` computes it in 64 bits, apart from both.
"""
import math

import torch

own = False

_kept = {}


def listed():
    return [
        # the likelihood of a single token: latency and the weight's bytes
        {"name": "loss_token", "op": "loss", "rows": 1, "vocab": 32768, "hidden": 4096, "topk": 0, "grad": False},
        # a few requests scored, a vocabulary of odd size
        {"name": "loss_requests", "op": "loss", "rows": 16, "vocab": 128003, "hidden": 2048, "topk": 0, "grad": False},
        # evaluation of a batch of text
        {"name": "loss_batch", "op": "loss", "rows": 4096, "vocab": 131072, "hidden": 4096, "topk": 0, "grad": False},
        # the last step of a training batch: the loss and both gradients
        {"name": "loss_train", "op": "loss", "rows": 4096, "vocab": 131072, "hidden": 4096, "topk": 0, "grad": True},
        # the same for a ragged batch and odd widths
        {"name": "loss_train_ragged", "op": "loss", "rows": 1000, "vocab": 32003, "hidden": 1028, "topk": 0, "grad": True},
        # a student against a teacher's 32 best tokens: how far it is
        {"name": "distill_batch", "op": "loss", "rows": 2048, "vocab": 32768, "hidden": 4096, "topk": 32, "grad": False},
        # and its training step, with 64 of them
        {"name": "distill_train", "op": "loss", "rows": 2048, "vocab": 50001, "hidden": 2048, "topk": 64, "grad": True},
        # sixteen tokens with eight experts each: most groups have a row or two
        {"name": "grouped_decode", "op": "grouped_nt", "rows": 128, "groups": 64, "n": 1536, "k": 4096, "tail": 0},
        # a prompt's tokens on eight experts each
        {"name": "grouped_prompt", "op": "grouped_nt", "rows": 32768, "groups": 64, "n": 1536, "k": 4096, "tail": 0},
        # odd sizes, and rows behind the last group
        {"name": "grouped_ragged", "op": "grouped_nt", "rows": 1003, "groups": 16, "n": 1540, "k": 4100, "tail": 21},
        # the gradient of the experts' rows in a training step
        {"name": "grouped_input_grad", "op": "grouped_nn", "rows": 16384, "groups": 64, "n": 4096, "k": 1536, "tail": 0},
        # and of their weights
        {"name": "grouped_weight_grad", "op": "grouped_tn", "rows": 16384, "groups": 64, "n": 1536, "k": 4096, "tail": 0},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v // step, -(-lo // step)), hi // step) * step


def draw(rng):
    op = rng.choice(["loss", "loss", "loss", "grouped_nt", "grouped_nt", "grouped_nn", "grouped_tn"])
    step = rng.choice([1, 8, 8, 64])     # odd sizes, whole 16-byte chunks, whole matrix-core steps
    if op == "loss":
        hidden = _log(rng, 64, 4096, step)
        vocab = _log(rng, 1000, 131072, rng.choice([1, 64]))
        return {"op": op, "rows": _log(rng, 1, 4096), "vocab": vocab, "hidden": hidden,
                "topk": rng.choice([0, 0, _log(rng, 1, 64)]), "grad": rng.random() < 0.5}
    groups = _log(rng, 1, 64)
    n, k = _log(rng, 64, 4096, step), _log(rng, 64, 4096, step)
    if groups * n * k > 64 * 1536 * 4096:
        n = max(step, 64 * 1536 * 4096 // (groups * k) // step * step)
    rows = _log(rng, 1, min(32768, 32768 * 1536 * 4096 // (n * k)))
    return {"op": op, "rows": rows, "groups": groups, "n": n, "k": k,
            "tail": rng.choice([0, 0, _log(rng, 1, 64)]) if op != "grouped_tn" else 0}


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "loss":
        m, v, k, top = case["rows"], case["vocab"], case["hidden"], case["topk"]
        # logits of a standard deviation of 2, and those of the target or the
        # teacher's first token up to 16 above: rows from sure to lost
        s["w"] = _normal(g, (v, k), 2.0 * k ** -0.5)
        none = torch.rand((m,), generator=g, device="cuda") < (1 / 9 if m > 1 else 0.0)
        if top == 0:
            t = torch.randint(0, v, (m,), generator=g, device="cuda")
            first = t
            s["targets"] = torch.where(none, -100, t)       # padding and prompt tokens
            s["scale"] = 1.0
        else:
            # distinct tokens, a row's list shorter here and there (-1)
            at = torch.randint(0, v, (m, 1), generator=g, device="cuda")
            by = torch.randint(1, v // top, (m, 1), generator=g, device="cuda")
            ids = (at + by * torch.arange(top, device="cuda")) % v
            first = ids[:, 0].contiguous()
            short = torch.rand((m, top), generator=g, device="cuda") < 0.1
            short[:, 0] = False
            s["ids"] = torch.where(short | none[:, None], -1, ids).to(torch.int32)
            fall = 0.5 * torch.rand((m, top), generator=g, device="cuda")
            s["teacher"] = 20.0 - torch.cumsum(fall, 1)
            s["scale"] = 0.5                                # temperature 2
        boost = 4.0 * torch.rand((m, 1), generator=g, device="cuda")
        s["x"] = (torch.randn((m, k), generator=g, device="cuda") + boost * s["w"][first].float()).bfloat16()
        if case["grad"]:
            if top == 0:
                # the mean over the rows that have a target
                s["dloss"] = torch.where(none, 0.0, 1.0 / (~none).sum().clamp(min=1)).float()
            else:
                # a weight for each row
                s["dloss"] = (torch.rand((m,), generator=g, device="cuda") + 0.5) * (4.0 / m)
        return s
    rows, e, n, k, op = (case[q] for q in ("rows", "groups", "n", "k", "op"))
    # each row's group by the groups' popularity, as a router leaves it
    host = torch.Generator().manual_seed(seed)
    p = torch.softmax(0.5 * torch.randn((e,), generator=host), 0)
    mine = torch.multinomial(p, rows - min(case["tail"], rows - 1), replacement=True, generator=host)
    sizes = torch.bincount(mine, minlength=e)
    s["largest"] = int(sizes.max())
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).cuda()
    s["a"] = _normal(g, (rows, n if op == "grouped_tn" else k))
    if op == "grouped_tn":
        s["b"] = _normal(g, (rows, k))
        s["c"] = None
    else:
        s["b"] = _normal(g, (e, n, k) if op == "grouped_nt" else (e, k, n), k ** -0.5)
        # (rows behind the last group stay as they are)
        s["c"] = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda") if case["tail"] else None
    return s


def _workspace(lib):
    """The process's one workspace, as a program that makes these calls in turn keeps it."""
    if "workspace" not in _kept:
        _kept["workspace"] = lib.Workspace()
    return _kept["workspace"]


def _run_own(s):
    import dense_gemm_05_amd as lib
    case, ws = s["case"], _workspace(lib)
    if case["op"] == "loss":
        x, w, scale = s["x"], s["w"], s["scale"]
        if case["topk"] == 0:
            loss, lse = lib.linear_cross_entropy(x, w, s["targets"], scale=scale, workspace=ws)
            if not case["grad"]:
                return loss, lse
            dx, dw = lib.linear_cross_entropy_backward(s["dloss"], x, w, s["targets"], lse, scale=scale, workspace=ws)
        else:
            loss, lse = lib.linear_distill(x, w, s["ids"], s["teacher"], scale=scale, workspace=ws)
            if not case["grad"]:
                return loss, lse
            dx, dw = lib.linear_distill_backward(s["dloss"], x, w, s["ids"], s["teacher"], lse, scale=scale,
                                                 workspace=ws)
        return loss, dx, dw
    if case["op"] == "grouped_nt":
        return lib.gemm_bf16_grouped_nt(s["a"], s["b"], s["offsets"], C=s["c"], workspace=ws)
    if case["op"] == "grouped_nn":
        return lib.gemm_bf16_grouped(s["a"], s["b"], s["offsets"], C=s["c"], workspace=ws)
    return lib.gemm_bf16_grouped_tn(s["a"], s["b"], s["offsets"], workspace=ws)


def _plain_loss(s):
    case, x, w = s["case"], s["x"].float(), s["w"].float()
    v = case["vocab"]
    z = (x @ w.t()).mul_(s["scale"])
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp_().sum(1, keepdim=True).log() + top
    if case["topk"] == 0:
        t = s["targets"][:, None]
        has = (t >= 0) & (t < v)
        ids, q = t.clamp(0, v - 1), has.float()
        some = has
        loss = torch.where(has, lse - z.gather(1, ids), 0.0)[:, 0]
    else:
        has = (s["ids"] >= 0) & (s["ids"] < v)
        ids = s["ids"].long().clamp(0, v - 1)
        some = has.any(1, keepdim=True)
        t = torch.where(has, s["teacher"] * s["scale"], -math.inf)
        t = t - torch.where(some, t.amax(1, keepdim=True), 0.0)
        e = t.exp()
        total = torch.where(some, e.sum(1, keepdim=True), 1.0)
        q = e / total
        loss = torch.where(has, q * (t - total.log() - z.gather(1, ids) + lse), 0.0).sum(1)
    if not case["grad"]:
        return loss, lse[:, 0]
    d = (z - lse).exp_().mul_(some.float())
    d.scatter_add_(1, ids, -q)
    d.mul_(s["dloss"][:, None] * s["scale"])
    return loss, (d @ w).bfloat16(), (d.t() @ x).bfloat16()


def _padded(s, t):
    """The groups' rows one behind the other to equal length, zeros behind them: [groups, largest, columns]."""
    first, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    row = first + torch.arange(s["largest"], device=t.device)
    has = row < end
    return torch.where(has[..., None], t[torch.where(has, row, 0)].float(), 0.0)


def _plain_grouped(s):
    op, a = s["case"]["op"], _padded(s, s["a"])
    if op == "grouped_tn":
        return torch.bmm(a.transpose(1, 2), _padded(s, s["b"]))
    b = s["b"].float()
    c = torch.bmm(a, b.transpose(1, 2) if op == "grouped_nt" else b)
    # each row's place among the padded ones
    rows = torch.arange(s["a"].shape[0], device=a.device)
    group = torch.searchsorted(s["offsets"][1:], rows.to(torch.int32), right=True)
    last = s["case"]["groups"] - 1
    at = (rows - s["offsets"].long()[group.clamp(max=last)]).clamp(max=s["largest"] - 1)
    c = c[group.clamp(max=last), at]
    return torch.where((group <= last)[:, None], c, 0.0).bfloat16()


def run(state):
    if own:
        return _run_own(state)
    return _plain_loss(state) if state["case"]["op"] == "loss" else _plain_grouped(state)


def work(case):
    if case["op"] == "loss":
        m, v, k = case["rows"], case["vocab"], case["hidden"]
        once = 2 * (m * k + v * k) + 8 * m * max(1, case["topk"]) + 8 * m
        # the gradient: the logits again, and two products of their size
        return {"bytes": once + (2 * (m * k + v * k) if case["grad"] else 0),
                "flops": (8 if case["grad"] else 2) * m * v * k}
    rows, e, n, k = (case[q] for q in ("rows", "groups", "n", "k"))
    rows -= min(case["tail"], rows - 1)
    if case["op"] == "grouped_tn":
        return {"bytes": 2 * rows * (n + k) + 4 * e * n * k, "flops": 2 * rows * n * k}
    used = e * (1.0 - (1.0 - 1.0 / e) ** rows)      # groups that have rows, in the mean
    return {"bytes": 2 * rows * (n + k) + 2 * used * n * k, "flops": 2 * rows * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "loss":
        o = s["offsets"].tolist()
        a, b = s["a"].double(), s["b"]
        if case["op"] == "grouped_tn":
            b = b.double()
            return torch.stack([torch.mm(a[i:j].t(), b[i:j]) for i, j in zip(o, o[1:])])
        c = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=a.device)
        for e, (i, j) in enumerate(zip(o, o[1:])):
            if j > i:
                w = b[e].double()
                c[i:j] = torch.mm(a[i:j], w.t() if case["op"] == "grouped_nt" else w)
        return c
    x, w = s["x"].double(), s["w"].double()
    logp = torch.mm(x, w.t()) * s["scale"]
    lse = torch.logsumexp(logp, 1)
    logp -= lse[:, None]
    target = torch.zeros((case["rows"], case["vocab"]), dtype=torch.float64, device=x.device)
    if case["topk"] == 0:
        row = torch.nonzero(s["targets"] >= 0)[:, 0]
        target[row, s["targets"][row]] = 1.0
        loss = -(target * logp).sum(1)
    else:
        t = (s["teacher"].double() * s["scale"]).masked_fill(s["ids"] < 0, -math.inf)
        q = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)
        row, slot = torch.nonzero(s["ids"] >= 0, as_tuple=True)
        target[row, s["ids"][row, slot].long()] = q[row, slot]
        loss = torch.special.xlogy(q, q).sum(1) - (target * logp).sum(1)
    if not case["grad"]:
        return loss, lse
    some = target.sum(1, keepdim=True) > 0
    d = (torch.exp(logp) * some - target) * (s["dloss"].double()[:, None] * s["scale"])
    return loss, torch.mm(d, w), torch.mm(d.t(), x)
