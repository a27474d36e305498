"""Routing by scores with a balance bias and groups, and activation checkpoints in 8 bits, as measured cases.

Operators: ``route`` (softmax or sigmoid scores, bias, groups -> experts, weights, pair lists; where the case says so
with the update of the bias that follows it in training), ``grad`` (gradient of the logits under sigmoid scores, from
the routing weights and the balance loss), ``checkpoint`` (activation rows to 8-bit codes with a scale per 128 columns,
and back), ``score`` (the selection's score of every pair from 8-bit rows) and ``compact`` (the weighted rows of the
retained pairs from 8-bit rows).

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the library's calls.
Sizes are those of the one-GPU expert shares of this repository's benchmark (32768 tokens, 128 experts, top-8,
16 local experts, hidden 2048, expert width 768; the wider share's expert width 1408) and generic smaller, odd and
ragged ones.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
FLT_MAX = 3.4028234663852886e38
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GROUP = 128  # columns that share one scale of an 8-bit row
SCALE = 2.5  # factor of the routing weights
RATE = 1e-3  # of the bias update


def listed():
    return [
        # one token of a decoding step: latency only
        {"name": "route_token", "op": "route", "T": 1, "E": 128, "K": 8, "dtype": "f32", "first": 0, "local": 128,
         "score": "sigmoid", "bias": True, "update": False, "groups": 1, "top": 1, "best": 1, "renorm": True,
         "masked": 0.0},
        # a training micro-batch of 32768 tokens, balanced by the bias, which is updated behind it
        {"name": "route_share", "op": "route", "T": 32768, "E": 128, "K": 8, "dtype": "f32", "first": 0, "local": 128,
         "score": "sigmoid", "bias": True, "update": True, "groups": 1, "top": 1, "best": 1, "renorm": True,
         "masked": 0.0},
        # experts in groups of 20, an odd number of tokens with padding, bf16, one GPU's part of the experts
        {"name": "route_groups", "op": "route", "T": 20011, "E": 160, "K": 6, "dtype": "bf16", "first": 40, "local": 21,
         "score": "sigmoid", "bias": True, "update": True, "groups": 8, "top": 3, "best": 2, "renorm": False,
         "masked": 0.15},
        # the backward of a training micro-batch: routing weights and the balance loss of packed sequences
        {"name": "grad_share", "op": "grad", "T": 32768, "E": 128, "K": 8, "dtype": "f32", "S": 8, "renorm": True,
         "masked": 0.0},
        # a small odd batch, weights that are not renormalised, bf16 logits, padding
        {"name": "grad_odd", "op": "grad", "T": 4099, "E": 61, "K": 3, "dtype": "bf16", "S": 5, "renorm": False,
         "masked": 0.1},
        # the [gate | up] rows of one GPU's expert share, kept in 8 bits from the forward to the backward
        {"name": "checkpoint_share", "op": "checkpoint", "rows": 262144, "width": 1536, "parts": 2, "dtype": "bf16"},
        # the input rows of a small fp32 layer, whose last group of columns is short
        {"name": "checkpoint_odd", "op": "checkpoint", "rows": 999, "width": 520, "parts": 1, "dtype": "f32"},
        # the score of every pair of the share from its 8-bit rows
        {"name": "score_share", "op": "score", "T": 32768, "K": 8, "E": 16, "D": 2048, "F": 768, "swiglu": True,
         "dtype": "bf16"},
        # a small fp32 layer of odd sizes
        {"name": "score_odd", "op": "score", "T": 1023, "K": 3, "E": 5, "D": 264, "F": 136, "swiglu": True,
         "dtype": "f32"},
        # the weighted rows of the share's retained pairs
        {"name": "compact_share", "op": "compact", "T": 32768, "K": 8, "E": 16, "F": 768, "swiglu": True,
         "dtype": "bf16", "rho": 0.6},
        # the same over the wider share's rows, few tokens and a quarter of the pairs
        {"name": "compact_odd", "op": "compact", "T": 2049, "K": 4, "E": 7, "F": 1408, "swiglu": True, "dtype": "bf16",
         "rho": 0.25},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route", "grad", "checkpoint", "score", "compact"])
    if op == "checkpoint":
        parts = rng.choice([1, 2])
        width = parts * 8 * _log_int(rng, 1, 512)
        return {"op": op, "rows": _log_int(rng, 1, min(262144, 400_000_000 // width // 2)), "width": width,
                "parts": parts, "dtype": rng.choice(["f32", "bf16"])}
    if op in ("score", "compact"):
        K, F = rng.randint(1, 10), 8 * _log_int(rng, 1, 256)
        case = {"op": op, "T": _log_int(rng, 1, min(32768, 180_000_000 // (K * F))), "K": K, "E": rng.randint(K, 64),
                "F": F, "swiglu": rng.random() < 0.8, "dtype": rng.choice(["f32", "bf16"])}
        if op == "score":
            case["D"] = 8 * rng.randint(1, 256)
        else:
            case["rho"] = rng.choice([1.0, 0.6, 0.25])
        return case
    groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
    E = groups * _log_int(rng, 2 if groups > 1 else 4, 512 // groups)
    top = rng.randint(1, groups)
    case = {"op": op, "T": _log_int(rng, 1, min(60000, 8_000_000 // E)), "E": E,
            "K": rng.randint(1, min(16, E // groups * top)), "dtype": rng.choice(["f32", "bf16"]),
            "masked": rng.choice([0.0, 0.2]), "renorm": rng.random() < 0.5}
    if op == "route":
        case["first"] = rng.choice([0, rng.randrange(E)])
        case["local"] = E - case["first"] if rng.random() < 0.5 else rng.randint(1, E - case["first"])
        case.update(score=rng.choice(["sigmoid", "sigmoid", "softmax"]), bias=rng.random() < 0.7, groups=groups, top=top,
                    best=rng.randint(1, 2))
        case["update"] = case["bias"] and rng.random() < 0.5
    else:
        case["S"] = rng.choice([1, rng.randint(2, 64)])
    return case


# ------------------------------------------------------------------------------------------------- inputs

def _router_inputs(case, gen):
    T, E = case["T"], case["E"]
    skew = torch.randn(E, generator=gen, device=DEV) * 0.8  # some experts are liked by every token
    x = (torch.randn(T, E, generator=gen, device=DEV) * 1.5 + skew).to(TYPES[case["dtype"]])
    mask = None
    if case["masked"]:
        mask = (torch.rand(T, generator=gen, device=DEV) >= case["masked"]).to(torch.uint8)
    return x, mask, skew


def _layer_inputs(case, gen):
    """Pairs of a routed layer, expert-major: their tokens, weights and segment ends, and the rows that a forward saves,
    some columns of which are much larger than the others."""
    T, E, K = case["T"], case["E"], case["K"]
    x = torch.randn(T, E, generator=gen, device=DEV)
    x[:, 0] += 1.0
    chosen = torch.sort(x, dim=1, descending=True).indices[:, :K]
    order = torch.argsort(chosen.reshape(-1), stable=True)
    width = case["F"] * (2 if case["swiglu"] else 1)
    spread = torch.exp(torch.randn(width, generator=gen, device=DEV) * 0.7)
    H = (torch.randn(T * K, width, generator=gen, device=DEV) * spread).to(TYPES[case["dtype"]])
    return {"tok": (order // K).int(), "counts": torch.bincount(chosen.reshape(-1), minlength=E).cpu(), "H": H,
            "alpha": torch.softmax(x, 1).gather(1, chosen).reshape(-1)[order].contiguous()}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if own:
        import load_recalibrated_expert_amd as lr
        s["lr"] = lr
        kind = lr.BF16 if case["dtype"] == "bf16" else lr.F32
    if op in ("route", "grad"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"], s["mask"], skew = _router_inputs(case, gen)
        if own:
            s["r"] = lr.Router(T=T, E=E, K=K, dtype=kind, first=case.get("first", 0), local=case.get("local", E),
                               renorm=case["renorm"], scale=SCALE, score=case.get("score", "sigmoid"),
                               groups=case.get("groups", 1), top_groups=case.get("top", 1),
                               group_best=case.get("best", 1), device=DEV)
        if op == "route":
            # what many updates have left: most of the experts' lead, in steps of the rate
            s["bias"] = torch.round(-skew / (6 * RATE)) * RATE if case["bias"] else None
            zero = lambda *d, t=torch.int32: torch.zeros(*d, dtype=t, device=DEV)  # noqa: E731
            # pair rows behind the last pair stay as they are: zeros here
            s["out"] = {"idx": zero(T, K), "w": zero(T, K, t=torch.float32), "counts": zero(E),
                        "seg_off": zero(case["local"] + 1, t=torch.int64), "tok": zero(T * K), "slot": zero(T * K),
                        "alpha": zero(T * K, t=torch.float32), "pmap": zero(T, K)}
            return s
        x = _clean(s["logits"], s["mask"])
        top, order = torch.sort(x, dim=1, descending=True, stable=True)
        s["idx"] = torch.where(top[:, :K] > -math.inf, order[:, :K], -1).int()
        live = s["idx"].view(-1) >= 0
        n = int(live.sum())
        s["pmap"] = torch.full((T * K,), -1, dtype=torch.int32, device=DEV)
        s["pmap"][live] = torch.randperm(n, generator=gen, device=DEV).int()
        s["pmap"] = s["pmap"].view(T, K)
        s["dalpha"] = torch.randn(max(n, 1), generator=gen, device=DEV)
        s["gloss"] = torch.full((1,), 0.75, device=DEV)
        S = case["S"]
        cut = torch.sort((torch.rand(S - 1, generator=gen, device=DEV) * (T + 1)).long().clamp(max=T)).values
        off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
        seq = _sequence_of(off, T)
        place = torch.where(s["idx"] >= 0, seq[:, None] * E + s["idx"], S * E).view(-1)
        counts = torch.bincount(place, minlength=S * E + 1)[:-1].view(S, E).int()
        many = torch.bincount(seq[x.amax(1) > -math.inf], minlength=S).double()
        norm = torch.where(many > 0, 0.01 * E / (K * (many > 0).sum().clamp(min=1) * many.clamp(min=1) ** 2), 0.0)
        s["balance"] = {"counts": counts, "norm": norm.float()}
        s["seq_off"] = off if S > 1 else None
    elif op == "checkpoint":
        spread = torch.exp(torch.randn(case["width"], generator=gen, device=DEV) * 0.7)
        s["rows"] = (torch.randn(case["rows"], case["width"], generator=gen, device=DEV) * spread).to(
            TYPES[case["dtype"]])
    else:
        s.update(_layer_inputs(case, gen))
        s["parts"] = 2 if case["swiglu"] else 1
        s["q"], s["scale"] = _quantise(s.pop("H"), s["parts"])
        counts, N = s.pop("counts").numpy(), case["T"] * case["K"]
        seg = np.concatenate([[0], np.cumsum(counts)])
        quota = counts
        if op == "score":
            s["G"] = torch.randn(case["T"], case["D"], generator=gen, device=DEV).to(TYPES[case["dtype"]])
        else:  # a budget of pairs over all experts; each keeps some of its own, in ascending order
            kept = math.ceil(case["rho"] * N)
            s["sel"] = torch.sort(torch.randperm(N, generator=gen, device=DEV)[:kept]).values.int()
            quota = np.diff(np.searchsorted(s["sel"].cpu().numpy(), seg))
        if own:
            s["p"] = lr.Problem(E=case["E"], T=case["T"], K=case["K"], D=case.get("D", 8), F=case["F"],
                                swiglu=case["swiglu"], seg_off=seg, quota=quota, device=DEV, dtype=kind)
            s["H"] = lr.Checkpoint(s["q"].contiguous(), s["scale"].contiguous())
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _clean(logits, mask):
    """f32 logits with NaN and masked tokens at -inf and +inf at the largest finite value."""
    x = logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=FLT_MAX)
    return x if mask is None else torch.where(mask[:, None] != 0, x, -math.inf)


def _shares(x):
    """Scores of -inf or finite logits divided by their sum over a row, in f32: softmax."""
    top = x.amax(1, keepdim=True)
    z = torch.where(x > -math.inf, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
    return z / z.sum(1, keepdim=True).clamp(min=1e-30)


def _sigmoid_shares(x):
    """The same for sigmoid scores: each over the row's largest exp(min(x, 0)), so that no sum is 0."""
    low = x.clamp(max=0)
    top = low.amax(1, keepdim=True)
    z = torch.exp(low - torch.where(top > -math.inf, top, 0.0)) / (1 + torch.exp(-x.abs()))
    z = torch.where(x > -math.inf, z, 0.0)
    return z / z.sum(1, keepdim=True).clamp(min=1e-30)


def _sigmoid(x):
    return torch.exp(x.clamp(max=0)) / (1 + torch.exp(-x.abs()))


def _route(s, case):
    T, E, K, o = case["T"], case["E"], case["K"], s["out"]
    x = _clean(s["logits"], s["mask"])
    # choices are whole numbers: the scores that decide them are in 64 bits
    d = x.double()
    if case["score"] == "sigmoid":
        c = 1 / (1 + torch.exp(-d))
    else:
        top = d.amax(1, keepdim=True)
        c = torch.exp(d - torch.where(top > -math.inf, top, 0.0))
        c = c / c.sum(1, keepdim=True).clamp(min=1e-300)
    if case["bias"]:
        c = c + s["bias"].double()
    c = torch.where(x > -math.inf, c, -math.inf)
    G = case["groups"]
    if G > 1:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["best"]]
        of_group = torch.where(best > -math.inf, best, 0.0).sum(2)
        of_group = torch.where(best[:, :, 0] > -math.inf, of_group, -math.inf)
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        stays = torch.zeros(T, G, device=DEV).scatter_(1, kept, 1.0) > 0
        c = torch.where(stays[:, :, None], c.view(T, G, E // G), -math.inf).view(T, E)
    c, order = torch.sort(c, dim=1, descending=True, stable=True)
    idx = torch.where(c[:, :K] > -math.inf, order[:, :K], -1).int()
    xk = torch.where(idx >= 0, x.gather(1, idx.clamp(min=0).long()), -math.inf)
    if case["renorm"]:
        w = (_sigmoid_shares if case["score"] == "sigmoid" else _shares)(xk) * SCALE
    elif case["score"] == "sigmoid":
        w = _sigmoid(xk) * SCALE
    else:
        w = torch.where(idx >= 0, _shares(x).gather(1, idx.clamp(min=0).long()), 0.0) * SCALE
    flat = idx.view(-1).long()
    counts = torch.bincount(torch.where(flat < 0, E, flat), minlength=E + 1)[:E].int()
    e = flat - case["first"]
    here = (flat >= 0) & (e >= 0) & (e < case["local"])
    order = torch.argsort(torch.where(here, e, case["local"]), stable=True)
    rank = torch.arange(T * K, device=DEV)
    row = torch.empty_like(rank)
    row[order] = rank
    in_list = rank < here.sum()
    seg = torch.zeros(case["local"] + 1, dtype=torch.int64, device=DEV)
    seg[1:] = torch.cumsum(counts[case["first"]:case["first"] + case["local"]].long(), 0)
    out = {"idx": idx, "w": w, "counts": counts, "seg_off": seg,
           "tok": torch.where(in_list, (order // K).int(), o["tok"]),
           "slot": torch.where(in_list, (order % K).int(), o["slot"]),
           "alpha": torch.where(in_list, w.view(-1)[order], o["alpha"]),
           "pmap": torch.where(here, row, -1).int().view(T, K)}
    if case["update"]:  # up where the count is under the mean
        n = counts.long()
        out["bias"] = s["bias"] + RATE * torch.sign(n.sum() - E * n).float()
    return out


def _sequence_of(off, T):
    """Sequence of every token."""
    if off is None:
        return torch.zeros(T, dtype=torch.int64, device=DEV)
    return torch.searchsorted(off[1:].contiguous(), torch.arange(T, device=DEV), right=True)


def _grad(s, case):
    T, E = case["T"], case["E"]
    idx, logits = s["idx"], s["logits"]
    x = _clean(logits, s["mask"])
    chosen = idx >= 0
    place = idx.clamp(min=0).long()
    y = torch.where(chosen & (s["pmap"] >= 0), s["dalpha"][s["pmap"].clamp(min=0).long()], 0.0) * SCALE
    xk = torch.where(chosen, x.gather(1, place), -math.inf)
    if case["renorm"]:
        q = _sigmoid_shares(xk)
        at_k = q * _sigmoid(-xk) * (y - (q * y).sum(1, keepdim=True))
    else:
        at_k = _sigmoid(xk) * _sigmoid(-xk) * y
    at_k = torch.where(chosen, at_k, 0.0)
    dx = torch.zeros(T, E + 1, device=DEV).scatter_add_(1, torch.where(chosen, place, E), at_k)[:, :E]
    p = _sigmoid_shares(x)
    seq = _sequence_of(s["seq_off"], T)
    c = s["balance"]["counts"].float()[seq]
    away = torch.where(x > -math.inf, _sigmoid(-x), 0.0)
    dx = dx + (s["gloss"] * s["balance"]["norm"])[seq][:, None] * p * away * (c - (p * c).sum(1, keepdim=True))
    return {"dlogits": dx.to(logits.dtype)}


def _grouped(x, parts):
    """Rows [n, parts * w] as [n, parts, groups, 128], zeros behind w."""
    n, w = x.shape[0], x.shape[1] // parts
    groups = (w + GROUP - 1) // GROUP
    y = torch.zeros(n, parts, groups * GROUP, dtype=x.dtype, device=DEV)
    y[:, :, :w] = x.view(n, parts, w)
    return y.view(n, parts, groups, GROUP)


def _rows(y, width):
    """The inverse of _grouped."""
    n, parts = y.shape[:2]
    return y.reshape(n, parts, -1)[:, :, :width // parts].reshape(n, width)


def _quantise(x, parts):
    """Codes int8 [n, width] and scales bf16 [n, parts, groups]: the smallest bf16 number at or over the 127th part of
    the group's largest magnitude, and the nearest whole numbers of scales, ties to even."""
    y = _grouped(x.float(), parts)
    amax = y.abs().amax(3).double()
    near = (amax / 127).clamp(min=2.0 ** -126).bfloat16()
    above = (near.view(torch.int16) + 1).view(torch.bfloat16)
    scale = torch.where(near.double() * 127 < amax, above, near)
    # quotients next to a half are told apart in 64 bits
    q = torch.round(y.double() / scale.double()[..., None])
    return _rows(q.to(torch.int8), x.shape[1]), scale


def _values(q, scale):
    """What codes stand for, in f32 (exact: 8 bits times 8)."""
    return _rows(_grouped(q, scale.shape[1]).float() * scale.float()[..., None], q.shape[1])


def _phi(h, swiglu):
    if not swiglu:
        return h
    F = h.shape[1] // 2
    return h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]


def _checkpoint(s, case):
    q, scale = _quantise(s["rows"], case["parts"])
    return {"scale": scale, "rows": _values(q, scale).to(s["rows"].dtype)}


def _score(s, case):
    phi = _phi(_values(s["q"], s["scale"]), case["swiglu"])
    g = s["G"].double().square().sum(1)
    return {"R": (s["alpha"].double().square() * g[s["tok"].long()] * phi.square().sum(1, dtype=torch.float64)).float()}


def _compact(s, case):
    sel = s["sel"].long()
    phi = _phi(_values(s["q"][sel], s["scale"][sel]), case["swiglu"])
    return {"PhiW": (phi * s["alpha"][sel][:, None]).to(TYPES[case["dtype"]])}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        lr = s["lr"]
        if op == "route":
            o = lr.route(s["r"], s["logits"], mask=s["mask"], bias=s["bias"], out=s["out"])
            if case["update"]:
                return {**o, "bias": lr.bias_update(s["r"], s["bias"], o["counts"], RATE)}
            return o
        if op == "grad":
            return {"dlogits": lr.route_bwd(s["r"], s["logits"], s["idx"], dalpha=s["dalpha"], pmap=s["pmap"],
                                            balance=s["balance"], gloss=s["gloss"], mask=s["mask"],
                                            seq_off=s["seq_off"])}
        if op == "checkpoint":
            c = lr.checkpoint(s["rows"], parts=case["parts"])
            return {"scale": c.scale, "rows": lr.restore(c, dtype=s["rows"].dtype)}
        if op == "score":
            return {"R": lr.score_checkpoint(s["p"], s["G"], s["H"], s["alpha"], s["tok"])}
        return {"PhiW": lr.compact_checkpoint(s["p"], s["sel"], s["H"], s["alpha"])}
    if op == "route":
        return _route(s, case)
    if op == "grad":
        return _grad(s, case)
    if op == "checkpoint":
        return _checkpoint(s, case)
    return _score(s, case) if op == "score" else _compact(s, case)


# ------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "checkpoint":  # rows in, codes out; codes in, rows out; scales both times
        n, w = case["rows"], case["width"]
        scales = n * case["parts"] * math.ceil(w / case["parts"] / GROUP) * 2
        return {"bytes": 2 * (n * w * (size + 1) + scales), "flops": 6 * n * w}
    if op in ("score", "compact"):
        N, F = case["T"] * case["K"], case["F"]
        parts = 2 if case["swiglu"] else 1
        row = parts * (F + 2 * math.ceil(F / GROUP))  # codes and scales of one pair
        if op == "score":
            return {"bytes": case["T"] * case["D"] * size + N * (row + 12), "flops": 10 * N * F + 2 * case["T"] * case["D"]}
        kept = case["rho"] * N
        return {"bytes": kept * (row + F * size + 8), "flops": 10 * kept * F}
    T, E, K = case["T"], case["E"], case["K"]
    rows = T * E * size + (T if case["masked"] else 0)
    if op == "route":  # idx, w and pmap of every slot; tok, slot and alpha of the local pairs
        pairs = T * K * (1 - case["masked"]) * case["local"] / E
        return {"bytes": rows + 12 * T * K + 12 * pairs + 4 * E * (1 + case["bias"] + case["update"]) + 8 * (case["local"] + 1),
                "flops": T * E * (12 + K)}
    return {"bytes": rows + T * E * size + 12 * T * K + case["S"] * (4 * E + 12), "flops": 14 * T * E}


# ------------------------------------------------------------------------------------------------- 64 bits

def _rows64(s):
    """Logits as float64 numpy rows by the operator's rules."""
    x = s["logits"].double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, FLT_MAX))
    if s["mask"] is not None:
        x[s["mask"].cpu().numpy() == 0] = -np.inf
    return x


def _logistic64(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "checkpoint":
        q, scale = _codes64(s["rows"], case["parts"])
        return {"scale": scale, "rows": _rows(q * scale[..., None], case["width"])}
    if op in ("score", "compact"):
        return _pairs64(s, case)
    x = _rows64(s)
    return _exact_route(s, case, x) if op == "route" else _exact_grad(s, case, x)


def _codes64(rows, parts):
    y = _grouped(rows.double(), parts)
    m, e = torch.frexp(y.abs().amax(3) / 127)
    # 8 bits of mantissa, rounded up
    scale = (torch.ceil(m * 256) / 256 * ((e.long() + 1023) << 52).view(torch.float64)).clamp(min=2.0 ** -126)
    z = y / scale[..., None]
    q = torch.floor(z)
    z -= q
    q += (z > 0.5) | ((z == 0.5) & (q % 2 != 0))
    return q, scale


def _pairs64(s, case):
    F, N = case["F"], s["q"].shape[0]
    pick = s["sel"].long() if case["op"] == "compact" else torch.arange(N, device=DEV)
    out, step = [], 32768
    for a in range(0, len(pick), step):
        j = pick[a:a + step]
        h = s["q"][j].double()
        column = torch.arange(h.shape[1], device=DEV)
        part = column // F if case["swiglu"] else torch.zeros_like(column)
        h *= s["scale"].double()[j][:, part, (column - part * F) // GROUP]
        if case["swiglu"]:
            gate, up = h.split(F, dim=1)
            h = gate * torch.sigmoid(gate) * up
        if case["op"] == "compact":
            out.append((h * s["alpha"].double()[j][:, None]).float())
        else:
            grad = s["G"][s["tok"][j].long()].double()
            out.append(torch.linalg.vecdot(h, h) * torch.linalg.vecdot(grad, grad) * s["alpha"].double()[j] ** 2)
    return {"PhiW" if case["op"] == "compact" else "R": torch.cat(out)}


def _exact_route(s, case, x):
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    there = x > -np.inf
    live = there.any(1)
    if case["score"] == "sigmoid":
        score = _logistic64(x)
    else:
        score = np.exp(x - np.where(live, x.max(1), 0)[:, None])
        score /= np.where(live, score.sum(1), 1)[:, None]
    c = score + (s["bias"].double().cpu().numpy() if case["bias"] else 0)
    c[~there] = -np.inf
    if G > 1:
        ordered = -np.sort(-c.reshape(T, G, E // G), axis=2)
        of_group = ordered[:, :, 0].copy()
        if case["best"] == 2 and E // G > 1:
            second = ordered[:, :, 1]
            of_group += np.where(second > -np.inf, second, 0)
        place = np.argsort(np.argsort(-of_group, axis=1, kind="stable"), axis=1, kind="stable")
        c = np.where(np.repeat(place < case["top"], E // G, axis=1), c, -np.inf)
    order = np.argsort(-c, axis=1, kind="stable")[:, :K]
    ok = np.take_along_axis(c, order, 1) > -np.inf
    idx = np.where(ok, order, -1)
    w = np.where(ok, np.take_along_axis(score, order, 1), 0)
    if case["renorm"]:
        w = w / np.where(w.sum(1) > 0, w.sum(1), 1)[:, None]
    w = SCALE * w
    counts = np.bincount(idx[ok], minlength=E)
    tok, slot = np.zeros(T * K, np.int32), np.zeros(T * K, np.int32)
    alpha, pmap, seg = np.zeros(T * K), np.full((T, K), -1, np.int32), [0]
    for e in range(case["first"], case["first"] + case["local"]):
        t, k = np.nonzero(idx == e)  # by token
        a, b = seg[-1], seg[-1] + len(t)
        tok[a:b], slot[a:b], alpha[a:b], pmap[t, k] = t, k, w[t, k], np.arange(a, b)
        seg.append(b)
    out = {"idx": idx.astype(np.int32), "w": w, "counts": counts.astype(np.int32), "seg_off": np.array(seg), "tok": tok,
           "slot": slot, "alpha": alpha, "pmap": pmap}
    if case["update"]:
        out["bias"] = s["bias"].double().cpu().numpy() + RATE * ((counts * E < counts.sum()) * 1.0 - (counts * E > counts.sum()))
    return out


def _exact_grad(s, case, x):
    T, E, K = case["T"], case["E"], case["K"]
    idx, pm, d = s["idx"].cpu().numpy(), s["pmap"].cpu().numpy(), s["dalpha"].double().cpu().numpy()
    score = _logistic64(x)
    slope = score * (1 - score)  # of each score with respect to its own logit; 0 at -inf
    rows = np.arange(T)
    ds = np.zeros((T, E))  # gradient of the scores
    under, mean = np.zeros(T), np.zeros(T)
    y = np.where((idx >= 0) & (pm >= 0), d[np.maximum(pm, 0)], 0) * SCALE
    if case["renorm"]:
        for k in range(K):
            at = idx[:, k] >= 0
            under[at] += score[rows[at], idx[at, k]]
        for k in range(K):
            at = idx[:, k] >= 0
            mean[at] += score[rows[at], idx[at, k]] * y[at, k] / under[at]
    for k in range(K):
        at = idx[:, k] >= 0
        ds[rows[at], idx[at, k]] = (y[at, k] - mean[at]) / under[at] if case["renorm"] else y[at, k]
    off = [0, T] if s["seq_off"] is None else s["seq_off"].cpu().tolist()
    c, norm = s["balance"]["counts"].cpu().numpy(), s["balance"]["norm"].double().cpu().numpy() * float(s["gloss"])
    for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
        total = score[a:b].sum(1)
        total = np.where(total > 0, total, 1)
        ds[a:b] += norm[i] * (c[i] - ((score[a:b] @ c[i]) / total)[:, None]) / total[:, None]
    return {"dlogits": ds * slope}
