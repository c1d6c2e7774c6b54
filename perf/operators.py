"""The routed operators of the W4A16 product, as cases to time and to compare.

Four operators that stand beside the fused product of one packed linear:

  route   which experts serve a token, and with what weight: softmax or sigmoid scores, a balance bias that only
          chooses, groups of experts, the top k, weights of the scores alone (optionally renormalised)
  up      each token's row through the packed 4-bit weights of its k experts, with SwiGLU in the epilogue or without
  down    each (token, expert) row through its expert's packed weights, weighted and summed over the token's experts
  lora    the low-rank adapter of each row's request added to the output of a shared projection

`own` False: the plain form, elementary torch operations in 32 bits (scores that decide in 64), rounded once at the
end.  `own` True: the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step: nothing but latency
        {"name": "route decode 1 token", "op": "route", "tokens": 1, "experts": 64, "top_k": 8, "score": "softmax",
         "groups": 1, "keep_groups": 1, "group_top": 1, "bias": False, "renorm": True, "scale": 1.0, "dtype": "bf16"},
        # a ragged batch of prompts over a number of experts that is no power of two, logits in 32 bits
        {"name": "route 519 tokens, 60 experts", "op": "route", "tokens": 519, "experts": 60, "top_k": 4,
         "score": "softmax", "groups": 1, "keep_groups": 1, "group_top": 1, "bias": True, "renorm": False,
         "scale": 1.0, "dtype": "f32"},
        # a large prefill with many experts in groups, sigmoid scores and a balance bias
        {"name": "route 16384 tokens, 256 in 8 groups", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8,
         "score": "sigmoid", "groups": 8, "keep_groups": 4, "group_top": 2, "bias": True, "renorm": True,
         "scale": 2.5, "dtype": "bf16"},
        # decode: one token, 8 of 64 experts, gate|up with SwiGLU; bound by the chosen experts' packed words
        {"name": "up decode 1 token", "op": "up", "tokens": 1, "experts": 64, "top_k": 8, "k": 2048, "n": 2048,
         "group": 128, "act": "swiglu", "dtype": "bf16", "out": "bf16"},
        # a decode batch: nearly every expert is chosen, by about three tokens each
        {"name": "up batch 24", "op": "up", "tokens": 24, "experts": 64, "top_k": 8, "k": 2048, "n": 2048,
         "group": 128, "act": "swiglu", "dtype": "f16", "out": "f16"},
        # a prefill through 8 experts of the 7B layer's gate|up size
        {"name": "up prefill 2048", "op": "up", "tokens": 2048, "experts": 8, "top_k": 2, "k": 4096, "n": 22016,
         "group": 128, "act": "swiglu", "dtype": "bf16", "out": "bf16"},
        # decode: the 8 chosen rows back down and summed, 32-bit output
        {"name": "down decode 1 token", "op": "down", "tokens": 1, "experts": 64, "top_k": 8, "k": 1024, "n": 2048,
         "group": 128, "dtype": "f16", "out": "f32"},
        # a ragged batch, small groups of channels and an odd number of outputs
        {"name": "down batch 100, n 2049", "op": "down", "tokens": 100, "experts": 64, "top_k": 8, "k": 1024,
         "n": 2049, "group": 64, "dtype": "bf16", "out": "bf16"},
        # a prefill over many experts: a few hundred rows each
        {"name": "down prefill 4096", "op": "down", "tokens": 4096, "experts": 64, "top_k": 8, "k": 1024, "n": 2048,
         "group": 128, "dtype": "bf16", "out": "bf16"},
        # one request's token beside a 4096 x 4096 projection
        {"name": "lora decode 1 row", "op": "lora", "rows": 1, "adapters": 8, "rank": 16, "k": 4096, "n": 4096,
         "mixed": True, "ranks": False, "base": True, "dtype": "f16", "out": "f16"},
        # a decode batch of many requests, adapters of different ranks, beside the 7B layer's up projection
        {"name": "lora batch 64, 32 adapters", "op": "lora", "rows": 64, "adapters": 32, "rank": 64, "k": 4096,
         "n": 11008, "mixed": True, "ranks": True, "base": True, "dtype": "bf16", "out": "bf16"},
        # prompts of a few requests: long runs of rows of one adapter
        {"name": "lora prefill 4096", "op": "lora", "rows": 4096, "adapters": 6, "rank": 32, "k": 4096, "n": 4096,
         "mixed": False, "ranks": False, "base": True, "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "up", "down", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, experts // groups * keep))
        return {"op": op, "tokens": _log(rng, 1, 16384) if experts <= 256 else _log(rng, 1, 8192), "experts": experts,
                "top_k": top_k, "score": rng.choice(["softmax", "sigmoid"]), "groups": groups, "keep_groups": keep,
                "group_top": rng.choice([1, 2]), "bias": rng.random() < 0.6, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op in ("up", "down"):
        experts = _log(rng, 4, 128)
        group = rng.choice([64, 128, 128, 256])
        k = group * max(1, _log(rng, 128, 4096) // group)
        n = _log(rng, 16, 4096)
        top_k = rng.randint(1, min(8, experts))
        case = {"op": op, "tokens": _log(rng, 1, 4096), "experts": experts, "top_k": top_k, "k": k, "n": n,
                "group": group, "dtype": rng.choice(["bf16", "f16"]), "out": rng.choice(["bf16", "f16", "f32"])}
        if op == "up":
            case["act"] = rng.choice(["swiglu", "none"])
            case["n"] += case["n"] % 2
        return case
    return {"op": op, "rows": _log(rng, 1, 4096), "adapters": _log(rng, 1, 48), "rank": 8 * rng.randint(1, 8),
            "k": 8 * _log(rng, 16, 512), "n": _log(rng, 16, 11008 if rng.random() < 0.3 else 4096),
            "mixed": rng.random() < 0.5, "ranks": rng.random() < 0.5, "base": rng.random() < 0.7,
            "dtype": rng.choice(["bf16", "f16"]), "out": rng.choice(["bf16", "f16", "f32"])}


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device)


def prepare(case, seed):
    gen = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    gen.manual_seed(seed)
    dev = gen.device
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        # a gate's logits: some experts are liked more; a few are switched off for some tokens
        s["logits"] = (1.5 * _randn(gen, t, e) + 0.5 * _randn(gen, e)).to(dtype)
        if t >= 16:
            off = torch.rand(t, e, generator=gen, device=dev) < 0.01
            s["logits"].masked_fill_(off, -math.inf)
        s["bias"] = 0.05 * _randn(gen, e) if case["bias"] else None
        return s
    if case["op"] in ("up", "down"):
        t, e, top, k, n, g = (case[c] for c in ("tokens", "experts", "top_k", "k", "n", "group"))
        like = _randn(gen, t, e) + 0.5 * _randn(gen, e)
        top_v, ids = torch.topk(like, top, dim=1)
        ids = ids.to(torch.int32)
        if t >= 16:
            ids[t - t // 16:] = -1  # rows that pad the batch have no expert
        s["ids"] = ids.contiguous()
        # the longest run of rows of one expert: what a padded batched product has to hold
        s["capacity"] = max(1, int(torch.bincount(ids.flatten().long() + 1, minlength=e + 1)[1:].max()))
        rows = t if case["op"] == "up" else t * top
        # activations with a few outlier channels, as calibration meets them
        x = _randn(gen, rows, k)
        x *= 1.0 + 9.0 * (torch.rand(k, generator=gen, device=dev) < 0.01)
        s["x"] = x.to(dtype)
        s["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (e, n, k // 8), generator=gen, device=dev, dtype=torch.int32)
        step = 0.5 + torch.rand(e, n, k // g, generator=gen, device=dev)
        s["scales"] = (step * (0.2 / math.sqrt(k))).to(torch.float16)
        s["zeros"] = torch.randint(5, 11, (e, n, k // g), generator=gen, device=dev, dtype=torch.uint8)
        if case["op"] == "down":
            s["weights"] = torch.softmax(top_v, dim=1)
        return s
    m, a, r, k, n = (case[c] for c in ("rows", "adapters", "rank", "k", "n"))
    s["x"] = _randn(gen, m, k).to(dtype)
    s["a"] = (_randn(gen, a, r, k) / math.sqrt(k)).to(dtype)
    s["b"] = (_randn(gen, a, n, r) / math.sqrt(r)).to(dtype)
    if case["mixed"]:  # every row another request, a tenth of them without an adapter
        ids = torch.randint(0, a, (m,), generator=gen, device=dev)
        if m >= 8:
            ids[torch.rand(m, generator=gen, device=dev) < 0.1] = -1
    else:  # prompts one after another, each of one adapter, the last one without
        cuts, _ = torch.sort(torch.rand(m, generator=gen, device=dev))
        ids = (cuts * (a + 0.5)).long()
        ids[ids == a] = -1
    s["adapter"] = ids.to(torch.int32)
    s["ranks"] = torch.randint(1, r + 1, (a,), generator=gen, device=dev, dtype=torch.int32) if case["ranks"] else None
    s["scaling"] = 0.5 + torch.rand(a, generator=gen, device=dev)
    s["base"] = _randn(gen, m, n).to(DTYPES[case["out"]]) if case["base"] else None
    return s


def run(state):
    case = state["case"]
    if own:
        return _calls(case, state)
    return {"route": _route, "up": _up, "down": _down, "lora": _lora}[case["op"]](case, state)


def _calls(case, s):
    import weight_only_int4_stats_amd as awq

    if case["op"] == "route":
        return awq.awq_route_experts(s["logits"], case["top_k"], bias=s["bias"], score=case["score"],
                                     n_group=case["groups"], topk_group=case["keep_groups"],
                                     group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"])
    if case["op"] == "up":
        return awq.awq_w4a16_experts_up(s["x"], s["ids"], s["qweight"], s["scales"], s["zeros"], act=case["act"],
                                        out_dtype=DTYPES[case["out"]], group_size=case["group"])
    if case["op"] == "down":
        return awq.awq_w4a16_experts_down(s["x"], s["ids"], s["weights"], s["qweight"], s["scales"], s["zeros"],
                                          out_dtype=DTYPES[case["out"]], group_size=case["group"])
    return awq.awq_lora_add(s["x"], s["adapter"], s["a"], s["b"], base=s["base"], scaling=s["scaling"],
                            ranks=s["ranks"], out_dtype=DTYPES[case["out"]])


# ---- plain forms ---------------------------------------------------------------


def _route(case, s):
    t, e, g = case["tokens"], case["experts"], case["groups"]
    logits = s["logits"].double()  # a choice between close scores is decided in 64 bits
    usable = logits > -math.inf
    if case["score"] == "softmax":
        top = torch.where(usable.any(1, keepdim=True), logits.amax(1, keepdim=True), 0.0)
        p = torch.where(usable, torch.exp(logits - top), 0.0)
        score = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(usable, choice, -math.inf)
    if g > 1:
        by_group = choice.view(t, g, e // g)
        best = torch.sort(by_group, dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(t, g, dtype=torch.bool, device=logits.device)
        keep.scatter_(1, order[:, :case["keep_groups"]], True)
        choice = torch.where(keep[:, :, None], by_group, -math.inf).view(t, e)
    value, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    value, ids = value[:, :case["top_k"]], ids[:, :case["top_k"]]
    none = value == -math.inf
    w = torch.where(none, 0.0, torch.gather(score, 1, ids))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(none, -1, ids).to(torch.int32), (w * case["scale"]).float()


def _dequantized(q, scales, zeros, group):
    """[..., K/8] packed words -> [..., K] weights in 32 bits."""
    shifts = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    codes = ((q.unsqueeze(-1) >> shifts) & 15).flatten(-2).float()
    codes = codes.unflatten(-1, (-1, group))
    return ((codes - zeros.float().unsqueeze(-1)) * scales.float().unsqueeze(-1)).flatten(-2)


def _experts(case, s, rows):
    """rows [S, K] in 32 bits (one per slot) through each slot's expert: [S, N]."""
    e, n, k, g = case["experts"], case["n"], case["k"], case["group"]
    ids = s["ids"].flatten().long()
    slots = ids.numel()
    live = (ids >= 0).unsqueeze(1)
    if slots <= e // 2:  # few slots: only their experts' weights
        i = ids.clamp_min(0)
        w = _dequantized(s["qweight"][i], s["scales"][i], s["zeros"][i], g)
        return torch.where(live, torch.bmm(w, rows.unsqueeze(2)).squeeze(2), 0.0)
    w = _dequantized(s["qweight"], s["scales"], s["zeros"], g)
    order = torch.argsort(ids, stable=True)
    sorted_ids = ids[order]
    first = torch.searchsorted(sorted_ids, torch.arange(e, device=ids.device))
    place = torch.arange(slots, device=ids.device) - first[sorted_ids.clamp_min(0)]
    cap = s["capacity"]
    at = torch.where(sorted_ids >= 0, sorted_ids * cap + place, e * cap)  # slots without an expert: a row of their own
    padded = torch.zeros(e * cap + 1, k, device=rows.device)
    padded[at] = rows[order]
    y = torch.bmm(padded[:-1].view(e, cap, k), w.transpose(1, 2).contiguous()).view(e * cap, n)
    y = torch.cat([y, torch.zeros(1, n, device=y.device)])
    out = torch.empty(slots, n, device=rows.device)
    out[order] = y[at]
    return torch.where(live, out, 0.0)


def _up(case, s):
    rows = s["x"].float().repeat_interleave(case["top_k"], dim=0)
    y = _experts(case, s, rows)
    if case["act"] == "swiglu":
        gate, up = y.chunk(2, dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(DTYPES[case["out"]])


def _down(case, s):
    y = _experts(case, s, s["x"].float())
    y = y * s["weights"].reshape(-1, 1)
    return y.view(case["tokens"], case["top_k"], -1).sum(1).to(DTYPES[case["out"]])


def _lora(case, s):
    n_ad, r, k, n = case["adapters"], case["rank"], case["k"], case["n"]
    mine = s["adapter"].long().unsqueeze(1) == torch.arange(n_ad, device=s["x"].device)  # [rows, adapters]
    used = torch.ones(n_ad, r, dtype=torch.bool, device=s["x"].device)
    if s["ranks"] is not None:
        used = torch.arange(r, device=s["x"].device) < s["ranks"].unsqueeze(1)
    h = s["x"].float() @ s["a"].float().view(n_ad * r, k).t()
    h = torch.where((mine.unsqueeze(2) & used), h.view(-1, n_ad, r) * s["scaling"].view(1, -1, 1), 0.0)
    y = h.view(-1, n_ad * r) @ s["b"].float().transpose(1, 2).reshape(n_ad * r, n)
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(DTYPES[case["out"]])


# ---- the definitions in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "lora":
        x, y = s["x"].double(), torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=s["x"].device)
        for i in range(case["adapters"]):
            rows = (s["adapter"] == i).nonzero().flatten()
            if rows.numel() == 0:
                continue
            r = case["rank"] if s["ranks"] is None else int(s["ranks"][i])
            delta = (x[rows] @ s["a"][i, :r].double().t()) @ s["b"][i, :, :r].double().t()
            y[rows] = float(s["scaling"][i]) * delta
        return y if s["base"] is None else y + s["base"].double()
    top, group = case["top_k"], case["group"]
    ids = s["ids"].flatten()
    out = torch.zeros(ids.numel(), case["n"], dtype=torch.float64, device=ids.device)
    for i in range(case["experts"]):
        slots = (ids == i).nonzero().flatten()
        if slots.numel() == 0:
            continue
        b = s["qweight"][i].contiguous().view(torch.uint8)  # two codes a byte, the lower channel in the low half
        q = torch.stack([b % 16, b // 16], dim=2).reshape(case["n"], case["k"]).double()
        w = (q - s["zeros"][i].double().repeat_interleave(group, 1)) * s["scales"][i].double().repeat_interleave(group, 1)
        x = s["x"][slots // top if case["op"] == "up" else slots].double()
        out[slots] = x @ w.t()
    if case["op"] == "up":
        if case["act"] == "none":
            return out
        half = case["n"] // 2
        return out[:, :half] * torch.sigmoid(out[:, :half]) * out[:, half:]
    w = s["weights"].double().reshape(-1, 1)
    return (out * w).reshape(case["tokens"], top, case["n"]).sum(1)


def _exact_route(case, s):
    logits = s["logits"].double().cpu().numpy()
    t, e = logits.shape
    groups, size = case["groups"], e // case["groups"]
    off = np.isneginf(logits)
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            z = np.exp(logits - logits.max(axis=1, keepdims=True))
            score = z / z.sum(axis=1, keepdims=True)
        else:
            score = 1.0 / (1.0 + np.exp(-logits))
    score[off] = 0.0
    choice = score.copy() if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    choice[off] = -np.inf
    if groups > 1:
        members = np.sort(choice.reshape(t, groups, size), axis=2)[:, :, ::-1]
        value = members[:, :, :case["group_top"]].sum(axis=2)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1)
        choice[np.repeat(rank >= case["keep_groups"], size, axis=1)] = -np.inf
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :case["top_k"]]
    gone = np.isneginf(np.take_along_axis(choice, ids, axis=1))
    w = np.where(gone, 0.0, np.take_along_axis(score, ids, axis=1))
    if case["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return np.where(gone, -1, ids).astype(np.int32), w * case["scale"]


def work(case):
    """Each input read once and each output written once; of the experts' and adapters' weights, those that are used
    (expected over an even routing)."""
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        return {"bytes": t * e * size[case["dtype"]] + t * case["top_k"] * 8 + (4 * e if case["bias"] else 0),
                "flops": 20.0 * t * e}
    if case["op"] in ("up", "down"):
        t, e, top, k, n = (case[c] for c in ("tokens", "experts", "top_k", "k", "n"))
        live = t - t // 16 if t >= 16 else t
        chosen = e * (1.0 - (1.0 - top / e) ** live)
        cols = n // 2 if case.get("act") == "swiglu" else n
        weights = chosen * n * (k / 2 + 3.0 * k / case["group"])
        x_rows, y_rows = (t, t * top) if case["op"] == "up" else (t * top, t)
        return {"bytes": weights + x_rows * k * 2 + y_rows * cols * size[case["out"]] + t * top * 4,
                "flops": 2.0 * live * top * k * n}
    m, a, r, k, n = (case[c] for c in ("rows", "adapters", "rank", "k", "n"))
    mean_rank = (r + 1) / 2 if case["ranks"] else r
    chosen = a * (1.0 - (1.0 - 1.0 / a) ** m)
    return {"bytes": chosen * mean_rank * (k + n) * 2 + m * k * 2 + m * n * size[case["out"]] * (2 if case["base"] else 1),
            "flops": 2.0 * m * mean_rank * (k + n)}
