"""Workloads of the training-step operators: the vocabulary cross entropy over the ranks' weight pieces, the
mixture-of-experts gate with its balance loss, and dropout alone and behind an all-reduce.  Each has a plain form in
elementary torch operations (``own`` false) and the library's calls (``own`` true) on the same inputs.

Definitions that both sides share:
  * Vocabulary pieces and rank chunks: rank r of p holds rows [r*C, min((r+1)*C, V)), C = ceil(V / p).
  * Dropout: element e of the index space (offset + rank * rank_stride + i) uses half word e % 8 (low half of each
    32-bit word first) of the Philox4x32-10 block with counter (e // 8, 0) and key seed.  It is kept when that half
    word is at least t = rint(prob * 2^16), and then multiplied by scale / (1 - t / 2^16).
  * Gate: an expert whose logit is -inf is never chosen; a slot that finds no expert holds id -1 and weight 0; a token
    that is masked, or whose logits are all -inf, is not counted anywhere.
"""
import math

import torch

own = False

TOP = 2.2e12  # flops of the largest cross entropy


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one generated token is scored against a 32,000-row head in 8 pieces: the weights are read once
        {"name": "ce_one_token", "op": "ce", "tokens": 1, "d": 4096, "vocab": 32000, "p": 8, "train": False, "ignored": 0.0},
        # a unit-test sized model: launches and latency
        {"name": "ce_tiny", "op": "ce", "tokens": 5, "d": 64, "vocab": 1000, "p": 2, "train": True, "ignored": 0.0},
        # nothing divides anything: odd width, a vocabulary that the ranks share unevenly, padded tokens
        {"name": "ce_odd", "op": "ce", "tokens": 777, "d": 1001, "vocab": 50257, "p": 3, "train": True, "ignored": 0.2},
        # a training micro-batch of a 4096-wide decoder over 8 ranks: loss and both gradients
        {"name": "ce_train", "op": "ce", "tokens": 2048, "d": 4096, "vocab": 32000, "p": 8, "train": True, "ignored": 0.05},
        # evaluation of long sequences: the loss alone
        {"name": "ce_score", "op": "ce", "tokens": 8192, "d": 4096, "vocab": 32000, "p": 8, "train": False, "ignored": 0.0},
        # a few decoded tokens through a small router
        {"name": "gate_decode", "op": "gate", "tokens": 4, "experts": 8, "k": 2, "p": 1, "dt": "bf16", "train": False, "masked": 0.0, "norm": True},
        # the all-to-all's MoE layer: 8 ranks x 4096 tokens, top 2 of 64
        {"name": "gate_layer", "op": "gate", "tokens": 4096, "experts": 64, "k": 2, "p": 8, "dt": "bf16", "train": True, "masked": 0.05, "norm": True},
        # many small experts and long batches, the router's logits in 32 bits
        {"name": "gate_wide", "op": "gate", "tokens": 16384, "experts": 256, "k": 8, "p": 8, "dt": "f32", "train": True, "masked": 0.0, "norm": False},
        # a small activation, odd length, another mask on each rank
        {"name": "dropout_small", "op": "dropout", "n": 12293, "p": 2, "dt": "f32", "prob": 0.1, "residual": False, "each": True},
        # 4096 tokens x 4096 channels on each of 8 ranks, added to the residual stream
        {"name": "dropout_large", "op": "dropout", "n": 4096 * 4096, "p": 8, "dt": "bf16", "prob": 0.1, "residual": True, "each": True},
        # the 8 MiB-per-rank all-reduce of a row-parallel layer with dropout and residual, and its backward
        {"name": "reduce_8MiB", "op": "reduce", "n": 2097152, "p": 8, "dt": "f32", "prob": 0.1, "residual": True},
        # an odd number of ranks and elements, no residual, and its backward
        {"name": "reduce_odd", "op": "reduce", "n": 1000003, "p": 5, "dt": "bf16", "prob": 0.25, "residual": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "gate", "dropout", "reduce"])
    if op == "ce":
        train = rng.random() < 0.7
        while True:
            n, d, v = _log(rng, 1, 8192), _log(rng, 64, 4096), _log(rng, 200, 64000)
            if rng.random() < 0.7:
                d = -(-d // 64) * 64
            if (8 if train else 2) * n * d * v <= TOP:
                break
        return {"op": op, "tokens": n, "d": d, "vocab": v, "p": rng.choice([1, 2, 4, 8, 5, 16]), "train": train,
                "ignored": rng.choice([0.0, 0.1, 0.5])}
    if op == "gate":
        e = rng.choice([4, 8, 16, 60, 64, 128, 256, rng.randint(4, 256)])
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": e, "k": rng.randint(1, min(8, e)),
                "p": rng.choice([1, 2, 4, 8]), "dt": rng.choice(["bf16", "f32"]), "train": rng.random() < 0.7,
                "masked": rng.choice([0.0, 0.1]), "norm": rng.random() < 0.5}
    n, p = _log(rng, 1000, 4 << 20), rng.choice([1, 2, 4, 8, 5])
    if rng.random() < 0.5:
        n = -(-n // 64) * 64
    case = {"op": op, "n": n, "p": p, "dt": rng.choice(["bf16", "f32"]), "prob": round(rng.uniform(0.0, 0.6), 3),
            "residual": rng.random() < 0.5}
    if op == "dropout":
        case["each"] = rng.random() < 0.5
    return case


def work(case):
    if case["op"] == "ce":
        n, d, v = case["tokens"], case["d"], case["vocab"]
        # The logits are not kept between the loss and its gradient: the gradient's pass computes them again.
        flops = (8 if case["train"] else 2) * n * d * v
        return {"bytes": (2 if case["train"] else 1) * 2 * (n * d + v * d) + 4 * n + (3 if case["train"] else 2) * 4 * n, "flops": flops}
    size = 2 if case["dt"] == "bf16" else 4
    if case["op"] == "gate":
        t, e, k = case["tokens"] * case["p"], case["experts"], case["k"]
        fwd = t * e * size + t * k * 8 + (t if case["masked"] else 0) + 4 * e * case["p"]
        return {"bytes": fwd + (t * e * size + t * k * 4 if case["train"] else 0), "flops": 5 * t * e}
    n, p = case["n"], case["p"]
    rows = 2 * p + (p if case["residual"] else 0) + (2 * p if case["op"] == "reduce" else 0)
    return {"bytes": rows * n * size, "flops": p * n}


# ---------------------------------------------------------------- inputs
def _type(dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


def _sizes(vocab, p):
    c = -(-vocab // p)
    return [max(0, min(vocab, (r + 1) * c) - r * c) for r in range(p)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    like = lambda ts: [torch.empty_like(t) for t in ts]  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] == "ce":
        n, d, v, p = case["tokens"], case["d"], case["vocab"], case["p"]
        w = (randn(v, d) * d ** -0.5).to(torch.bfloat16)
        # frequent words come first, as a tokenizer's ranks have it
        y = (rand(n) ** 3 * v).long().clamp_(max=v - 1)
        # a partly trained head: the hidden state leans towards its own target
        wy = w[y].float()
        h = randn(n, d) + wy / wy.square().sum(1, keepdim=True).clamp_min(1e-6) * (8 * rand(n, 1))
        y[rand(n) < case["ignored"]] = -100
        count = (y >= 0).sum().clamp_min(1)
        s |= {"hidden": h.to(torch.bfloat16), "weight": [t.clone() for t in torch.split(w, _sizes(v, p))], "target": y.to(torch.int32),
              "dloss": (y >= 0).float() / count}
        s |= {"loss": torch.empty(n, device="cuda"), "lse": torch.empty(n, device="cuda")}
        if case["train"]:
            s |= {"dhidden": torch.empty_like(s["hidden"]), "dweight": like(s["weight"])}
        return s
    dt, p = _type(case["dt"]), case["p"]
    if case["op"] == "gate":
        t, e, k = case["tokens"], case["experts"], case["k"]
        liked = randn(e)  # some experts are more popular than others
        s["logits"] = [(1.5 * randn(t, e) + 0.5 * liked).to(dt) for _ in range(p)]
        s["mask"] = None
        if case["masked"]:
            s["mask"] = [(rand(t) >= case["masked"]).to(torch.uint8) for _ in range(p)]
        s["dweights"] = [randn(t, k) * 0.01 for _ in range(p)]
        s["dloss"] = torch.ones(1, device="cuda")
        s["coef"] = 0.01
        s["ids"] = [torch.empty(t, k, dtype=torch.int32, device="cuda") for _ in range(p)]
        s["weights"] = like(s["dweights"])
        s["counts"] = [torch.empty(e, dtype=torch.int32, device="cuda") for _ in range(p)]
        s["stats"] = torch.empty(2 * e + 1, device="cuda")
        s["loss"] = torch.empty(1, device="cuda")
        if case["train"]:
            s["dlogits"] = like(s["logits"])
        return s
    n = case["n"]
    s["x"] = [randn(n).to(dt) for _ in range(p)]
    # a row-parallel layer's ranks hold the same residual stream; otherwise each rank has its own
    s["residual"] = None
    if case["residual"]:
        base = randn(n).to(dt)
        s["residual"] = [base.clone() if case["op"] == "reduce" else randn(n).to(dt) for _ in range(p)]
    s["y"] = like(s["x"])
    s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda"))
    s["offset"] = 8 * int(torch.randint(0, 1 << 40, (1,), generator=g, device="cuda"))
    if case["op"] == "reduce":
        dy = randn(n).to(dt)
        s["dy"] = [dy.clone() for _ in range(p)]
        s["dx"] = like(s["x"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"ce": _plain_ce, "gate": _plain_gate, "dropout": _plain_dropout, "reduce": _plain_reduce}[case["op"]](s, case)


def _own(s, case):
    import collective_rc_all_b200 as rc

    if case["op"] == "ce":
        if "ws" not in s:  # a training program keeps one workspace for its step
            s["ws"] = torch.empty(rc.rc_vocab_ce_workspace(case["tokens"], case["d"], case["vocab"], case["p"], backward=case["train"]),
                                  dtype=torch.uint8, device="cuda")
        rc.rc_vocab_ce_forward(s["hidden"], s["weight"], s["target"], s["loss"], s["lse"], ignore_index=-100, workspace=s["ws"])
        out = {"loss": s["loss"], "lse": s["lse"]}
        if case["train"]:
            rc.rc_vocab_ce_backward(s["hidden"], s["weight"], s["target"], s["lse"], s["dloss"], s["dhidden"], s["dweight"],
                                    ignore_index=-100, workspace=s["ws"])
            out |= {"dhidden": s["dhidden"], "dweight": s["dweight"]}
        return out
    if case["op"] == "gate":
        if "ws" not in s:
            s["ws"] = torch.empty(rc.rc_moe_gate_workspace(case["tokens"], case["experts"], case["p"]), dtype=torch.uint8, device="cuda")
        rc.rc_moe_gate(s["logits"], s["ids"], s["weights"], s["counts"], s["stats"], s["loss"], token_mask=s["mask"],
                       normalize=case["norm"], coef=s["coef"], workspace=s["ws"])
        out = {"ids": s["ids"], "weights": s["weights"], "counts": s["counts"], "stats": s["stats"], "loss": s["loss"]}
        if case["train"]:
            rc.rc_moe_gate_backward(s["logits"], s["ids"], s["stats"], s["dlogits"], dweights=s["dweights"], dloss=s["dloss"],
                                    token_mask=s["mask"], normalize=case["norm"], coef=s["coef"])
            out["dlogits"] = s["dlogits"]
        return out
    if case["op"] == "dropout":
        rc.rc_dropout(s["x"], s["y"], case["prob"], s["seed"], offset=s["offset"], rank_stride=case["n"] if case["each"] else 0,
                      residual=s["residual"])
        return {"y": s["y"]}
    rc.rc_all_reduce_dropout(s["x"], s["y"], case["prob"], s["seed"], offset=s["offset"], residual=s["residual"])
    rc.rc_dropout(s["dy"], s["dx"], case["prob"], s["seed"], offset=s["offset"])
    return {"y": s["y"], "dx": s["dx"]}


def _plain_ce(s, case):
    h, w = s["hidden"].float(), torch.cat(s["weight"]).float()
    y = s["target"].long()
    live = y >= 0
    at = torch.where(live, y, 0)[:, None]
    z = h @ w.T
    top = z.amax(1, keepdim=True)
    lse = top + (z - top).exp().sum(1, keepdim=True).log()
    loss = torch.where(live, (lse - z.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if case["train"]:
        g = (z - lse).exp()
        g.scatter_add_(1, at, torch.full_like(lse, -1.0))
        g *= torch.where(live, s["dloss"], 0.0)[:, None]
        out["dhidden"] = (g @ w).to(torch.bfloat16)
        out["dweight"] = list(torch.split((g.T @ h).to(torch.bfloat16), _sizes(case["vocab"], case["p"])))
    return out


def _plain_gate(s, case):
    p, e, k = case["p"], case["experts"], case["k"]
    z = torch.stack(s["logits"]).float()
    live = z.amax(-1) > -math.inf
    if s["mask"] is not None:
        live &= torch.stack(s["mask"]) != 0
    prob = torch.where(live[..., None], torch.softmax(torch.where(live[..., None], z, 0.0), -1), 0.0)
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :k]
    found = live[..., None] & (z.gather(-1, order) > -math.inf)
    chosen = torch.zeros_like(z).scatter_(-1, order, found.float())
    counts = chosen.sum(1)
    picked = torch.where(found, prob.gather(-1, order), 0.0)
    share = picked.sum(-1, keepdim=True).clamp_min(1e-38)
    weights = picked / share if case["norm"] else picked
    m = live.sum().float()
    f, mean = counts.sum(0) / (k * m.clamp_min(1)), prob.sum((0, 1)) / m.clamp_min(1)
    loss = (s["coef"] * e * (f * mean).sum()).reshape(1)
    out = {"ids": list(torch.where(found, order, -1).int()), "weights": list(weights), "counts": list(counts.int()),
           "stats": torch.cat([f, mean, m.reshape(1)]), "loss": loss}
    if case["train"]:
        dw = torch.where(found, torch.stack(s["dweights"]), 0.0)
        if case["norm"]:
            dw = (dw - (dw * weights).sum(-1, keepdim=True)) / share
        dp = (s["dloss"] * s["coef"] * e * f / m.clamp_min(1)).expand_as(z).scatter_add(-1, order, torch.where(found, dw, 0.0))
        dz = prob * (dp - (prob * dp).sum(-1, keepdim=True))
        out["dlogits"] = list(dz.to(_type(case["dt"])))
    return out


def _philox(block, seed):
    """The four 32-bit words of Philox4x32-10 (Salmon et al., 2011) for each counter (block, 0), in 64-bit integers."""
    low = 0xFFFFFFFF
    a, b, c, d = block & low, (block >> 32) & low, torch.zeros_like(block), torch.zeros_like(block)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((y >> 32) & low) ^ b ^ k0, y & low, ((x >> 32) & low) ^ d ^ k1, x & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([a, b, c, d], -1)


def _kept(first, n, seed, prob):
    """Truth values of elements first .. first + n - 1; `first` is a multiple of 8."""
    block = first // 8 + torch.arange(-(-n // 8), device="cuda")
    words = _philox(block, seed)
    half = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:n]
    return half >= round(prob * 65536)


def _factor(prob):
    t = round(prob * 65536)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def _mask(s, case, first):
    n = case["n"]
    if first % 8 == 0:
        return _kept(first, n, s["seed"], case["prob"])
    return _kept(first - first % 8, n + first % 8, s["seed"], case["prob"])[first % 8:]


def _plain_dropout(s, case):
    x = torch.stack(s["x"]).float()
    stride = case["n"] if case["each"] else 0
    keep = torch.stack([_mask(s, case, s["offset"] + r * stride) for r in range(case["p"])])
    y = torch.where(keep, x * _factor(case["prob"]), 0.0)
    if s["residual"] is not None:
        y = torch.stack(s["residual"]).float() + y
    return {"y": list(y.to(_type(case["dt"])))}


def _plain_reduce(s, case):
    keep, dt = _mask(s, case, s["offset"]), _type(case["dt"])
    y = torch.where(keep, torch.stack(s["x"]).float().sum(0) * _factor(case["prob"]), 0.0).expand(case["p"], -1)
    if s["residual"] is not None:
        y = torch.stack(s["residual"]).float() + y
    dx = torch.where(keep, torch.stack(s["dy"]).float() * _factor(case["prob"]), 0.0)
    return {"y": list(y.to(dt)), "dx": list(dx.to(dt))}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        h = s["hidden"].double()
        w = torch.cat([t.double() for t in s["weight"]])
        y = s["target"].long()
        valid = torch.nonzero(y >= 0)[:, 0]
        z = torch.mm(h, w.t())
        lse = torch.logsumexp(z, 1)
        loss = torch.zeros_like(lse)
        loss[valid] = lse[valid] - z[valid, y[valid]]
        out = {"loss": loss, "lse": lse}
        if case["train"]:
            z.sub_(lse[:, None]).exp_()
            z[valid, y[valid]] -= 1
            scale = torch.zeros_like(lse)
            scale[valid] = s["dloss"].double()[valid]
            z.mul_(scale[:, None])
            out["dhidden"] = torch.mm(z, w)
            out["dweight"] = [torch.mm(piece.t(), h) for piece in torch.split(z, [len(t) for t in s["weight"]], dim=1)]
        return out
    if case["op"] == "gate":
        return _exact_gate(case, s)
    import numpy as np

    t = int(np.rint(case["prob"] * 65536))
    up = 65536.0 / (65536.0 - t)
    keep = []
    for r in range(case["p"]):
        first = s["offset"] + (r * case["n"] if case.get("each") else 0)
        e = np.arange(case["n"], dtype=np.uint64) + np.uint64(first)
        blocks, where = np.unique(e >> np.uint64(3), return_inverse=True)
        x0, x1 = blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32)
        x2 = x3 = np.zeros_like(x0)
        key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
        for _ in range(10):
            u, v = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = ((v >> np.uint64(32)) ^ x1 ^ np.uint64(key[0]), v & np.uint64(0xFFFFFFFF),
                              (u >> np.uint64(32)) ^ x3 ^ np.uint64(key[1]), u & np.uint64(0xFFFFFFFF))
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        lane = (e & np.uint64(7)).astype(np.int64)
        word = np.stack([x0, x1, x2, x3], 1)[where, lane // 2]
        keep.append(torch.from_numpy((word >> (16 * (lane % 2)).astype(np.uint64) & np.uint64(0xFFFF)) >= np.uint64(t)).cuda())
        if not case.get("each"):
            keep *= case["p"]
            break
    drop = lambda x, k: torch.where(k, x.double() * up, torch.zeros((), dtype=torch.float64, device="cuda"))  # noqa: E731
    extra = [0.0] * case["p"] if s["residual"] is None else [r.double() for r in s["residual"]]
    if case["op"] == "dropout":
        return {"y": [drop(x, k) + r for x, k, r in zip(s["x"], keep, extra)]}
    total = torch.zeros(case["n"], dtype=torch.float64, device="cuda")
    for x in s["x"]:
        total += x.double()
    return {"y": [drop(total, keep[0]) + r for r in extra], "dx": [drop(x, keep[0]) for x in s["dy"]]}


def _exact_gate(case, s):
    e, k, t = case["experts"], case["k"], case["tokens"]
    z = torch.cat(s["logits"]).double()
    live = torch.isfinite(z.max(1).values)
    if s["mask"] is not None:
        live = live & torch.cat(s["mask"]).bool()
    q = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) * live[:, None]
    # rank of each expert in its row: how many are larger, or equal with a lower index (a stable ascending sort of -z)
    first = torch.argsort(-z, dim=1, stable=True)[:, :k]
    w = q.gather(1, first)
    total = w.sum(1, keepdim=True)
    if case["norm"]:
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    m = float(live.sum())
    hits = torch.zeros_like(q).scatter_(1, first, 1.0) * live[:, None]
    f, mean = hits.sum(0) / (k * max(m, 1.0)), q.sum(0) / max(m, 1.0)
    out = {"ids": None, "weights": list(w.split(t)), "counts": None, "stats": torch.cat([f, mean, f.new_tensor([m])]),
           "loss": (s["coef"] * e * torch.dot(f, mean)).reshape(1)}
    if case["train"]:
        up = torch.cat(s["dweights"]).double() * live[:, None]
        slope = float(s["dloss"]) * s["coef"] * e / max(m, 1.0) * f
        grad = q * (slope - (q @ slope)[:, None])
        inner = (up * w).sum(1, keepdim=True)
        if case["norm"]:  # the chosen weights are a softmax over the chosen logits
            grad.scatter_add_(1, first, w * (up - inner))
        else:
            grad -= q * inner
            grad.scatter_add_(1, first, w * up)
        out["dlogits"] = list((grad * live[:, None]).split(t))
    return out
