"""The measured cases of two operators of the layer's surroundings: the expert choice of a router
(`route`) and the dense projection with its epilogue (`linear`).

`run` with `own` false computes them from elementary torch operations; with `own` true it calls
the library. Every case is built from its sizes and a seed alone."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # --- route ---
        # one token of a decode step over the layer's 16 experts: latency only
        dict(name="route_one", op="route", T=1, E=16, k=2, scoring="softmax", bias=False, G=1, tg=1,
             group_score="max", renorm=True, scale=1.0, masked=0.0, padded=0.0),
        # a fine-grained decode batch: 128 experts, 8 of them per token
        dict(name="route_fine_grained", op="route", T=256, E=128, k=8, scoring="softmax", bias=False, G=1,
             tg=1, group_score="max", renorm=True, scale=1.0, masked=0.0, padded=0.0),
        # odd sizes: five expert groups of 32, plain softmax weights, some experts switched off
        dict(name="route_odd", op="route", T=12345, E=160, k=6, scoring="softmax", bias=False, G=5, tg=3,
             group_score="max", renorm=False, scale=16.0, masked=0.02, padded=0.0),
        # a padded batch of grouped sigmoid routing with a balance bias
        dict(name="route_padded", op="route", T=4099, E=256, k=8, scoring="sigmoid", bias=True, G=8, tg=4,
             group_score="top2", renorm=True, scale=2.5, masked=0.0, padded=0.3),
        # a whole prompt chunk of the same
        dict(name="route_prompt", op="route", T=65536, E=256, k=8, scoring="sigmoid", bias=True, G=8, tg=4,
             group_score="top2", renorm=True, scale=2.5, masked=0.0, padded=0.0),
        # --- linear ---
        # single token, square projection with bias and residual: weight streaming and latency
        dict(name="linear_one", op="linear", T=1, K=4096, N=4096, act="none", w="bf16", bias=True,
             residual=True, pad=0),
        # the decode batch through a shared expert: gate_up with SiLU-and-mul, then down with E4M3
        # weights onto the residual
        dict(name="linear_decode_gate_up", op="linear", T=64, K=4096, N=11008, act="swiglu", w="bf16",
             bias=False, residual=False, pad=0),
        dict(name="linear_decode_down_e4m3", op="linear", T=64, K=11008, N=4096, act="none", w="e4m3",
             bias=False, residual=True, pad=0),
        # a small expert's gate_up at the fine-grained batch
        dict(name="linear_small_gate_up", op="linear", T=256, K=2048, N=768, act="swiglu", w="bf16",
             bias=True, residual=False, pad=0),
        # nothing divides a tile: odd rows and columns, x a slice of a wider buffer
        dict(name="linear_ragged", op="linear", T=777, K=2040, N=1531, act="gelu_tanh", w="bf16", bias=True,
             residual=True, pad=72),
        # a prompt through a shared expert
        dict(name="linear_prompt_gate_up", op="linear", T=4096, K=4096, N=14336, act="swiglu", w="bf16",
             bias=False, residual=False, pad=0),
        dict(name="linear_prompt_down_e4m3", op="linear", T=4096, K=14336, N=4096, act="none", w="e4m3",
             bias=False, residual=True, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST_FLOPS = 2 * 4096 * 4096 * 2 * 14336  # of the largest listed case


def draw(rng):
    if rng.random() < 0.4:
        G = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
        E = G * _log(rng, max(2, 8 // G), 384 // G)
        tg = rng.randint(1, G)
        k = min(_log(rng, 1, 16), E // G * tg)
        scoring = rng.choice(["softmax", "sigmoid"])
        return dict(op="route", T=_log(rng, 1, 65536 * 256 // max(E, 256)), E=E, k=k, scoring=scoring,
                    bias=rng.random() < 0.6, G=G, tg=tg, group_score=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    masked=rng.choice([0.0, 0.0, 0.05]), padded=rng.choice([0.0, 0.0, 0.25]))
    T, w = _log(rng, 1, 8192), rng.choice(["bf16", "bf16", "e4m3"])
    act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu"])
    K = 16 * _log(rng, 8, 1024) + (8 if w == "bf16" and rng.random() < 0.5 else 0)
    N = _log(rng, 64, 16384)
    most = _MOST_FLOPS // (2 * T * K * (2 if act == "swiglu" else 1))
    return dict(op="linear", T=T, K=K, N=max(1, min(N, most)), act=act, w=w, bias=rng.random() < 0.5,
                residual=rng.random() < 0.5, pad=rng.choice([0, 0, 8 if w == "bf16" else 16, 128]))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(case=case)
    T = case["T"]
    if case["op"] == "route":
        E = case["E"]
        s["logits"] = normal(T, E)
        if case["masked"]:  # experts that are switched off for a token
            s["logits"][torch.rand(T, E, generator=g, device=DEV) < case["masked"]] = -math.inf
        s["bias"] = 0.1 * normal(E) if case["bias"] else None
        # rows of padding, which no token stands behind
        s["mask"] = (torch.rand(T, generator=g, device=DEV) >= case["padded"]) if case["padded"] else None
        return s
    K, N = case["K"], case["N"]
    rows = 2 * N if case["act"] == "swiglu" else N
    s["x"] = normal(T, K + case["pad"]).bfloat16()[:, :K]
    W = 0.02 * normal(rows, K)
    if case["w"] == "e4m3":  # codes with one scale per row, the largest magnitude of a row at 448
        s["scale"] = (W.abs().amax(1) / 448.0).clamp_min(1e-12)
        s["W"] = (W / s["scale"][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["W"], s["scale"] = W.bfloat16(), None
    s["bias"] = normal(rows).bfloat16() if case["bias"] else None
    s["residual"] = normal(T, N).bfloat16() if case["residual"] else None
    return s


def _route_plain(s, c):
    logits, bias, mask = s["logits"].double(), s["bias"], s["mask"]
    ok = torch.isfinite(logits)
    if mask is not None:
        ok = ok & mask[:, None]
    logits = torch.where(ok, logits, -math.inf)
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = ex / ex.sum(1, keepdim=True)
    # without a bias the scores rank as the logits do
    rank_by_score = bias is not None or (c["G"] > 1 and c["group_score"] == "top2")
    choice = score if bias is None else score + bias.double()
    choice = torch.where(ok, choice if rank_by_score else logits, -math.inf)
    T, E, G = c["T"], c["E"], c["G"]
    if G > 1:
        inside = choice.view(T, G, E // G).sort(dim=-1, descending=True).values
        group = inside[:, :, 0]
        if c["group_score"] == "top2" and E // G > 1:
            second = inside[:, :, 1]
            group = group + torch.where(second > -math.inf, second, 0.0)
        kept = group.sort(dim=-1, descending=True, stable=True).indices[:, :c["tg"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=choice.device).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], choice.view(T, G, E // G), -math.inf).view(T, E)
    best, ids = choice.sort(dim=-1, descending=True, stable=True)
    best, ids = best[:, :c["k"]], ids[:, :c["k"]]
    live = best > -math.inf
    u = (ex if c["scoring"] == "softmax" and c["renorm"] else score).gather(1, ids)
    u = torch.where(live, u, 0.0)
    if c["renorm"]:
        total = u.sum(1, keepdim=True)
        u = u / torch.where(total > 0, total, 1.0)
    return torch.where(live, ids, -1).int(), (c["scale"] * u).float()


def _linear_plain(s, c):
    W = s["W"].float() if s["scale"] is None else s["W"].view(torch.float8_e4m3fn).float() * s["scale"][:, None]
    v = torch.matmul(s["x"].float(), W.t())
    if s["bias"] is not None:
        v = v + s["bias"].float()
    act = c["act"]
    if act == "swiglu":
        gate, up = v[:, :c["N"]], v[:, c["N"]:]
        v = gate / (1.0 + torch.exp(-gate)) * up
    elif act == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif act == "relu":
        v = v.clamp_min(0.0)
    elif act == "gelu":
        v = 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.bfloat16()


def run(state):
    c = state["case"]
    if own:
        import lora_mixture_experts_amd as ml

        if c["op"] == "route":
            return ml.route(state["logits"], c["k"], scoring=c["scoring"], bias=state["bias"], n_groups=c["G"],
                            topk_groups=c["tg"], group_score=c["group_score"], renormalize=c["renorm"],
                            scale=c["scale"], token_mask=state["mask"])
        return ml.linear(state["x"], state["W"], w_scale=state["scale"], bias=state["bias"], act=c["act"],
                         residual=state["residual"])
    return _route_plain(state, c) if c["op"] == "route" else _linear_plain(state, c)


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        # logits in, ids and weights out; a few operations for each score
        nbytes = 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0) + (T if case["padded"] else 0)
        return dict(bytes=nbytes, flops=8 * T * E)
    K, N = case["K"], case["N"]
    rows = 2 * N if case["act"] == "swiglu" else N
    nbytes = 2 * T * K + (rows * (K + 4) if case["w"] == "e4m3" else 2 * rows * K) + 2 * T * N
    nbytes += (2 * rows if case["bias"] else 0) + (2 * T * N if case["residual"] else 0)
    return dict(bytes=nbytes, flops=2 * T * K * rows)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        W = s["W"].double() if s["scale"] is None else s["W"].view(torch.float8_e4m3fn).double()
        z = s["x"].double() @ W.T
        del W
        if s["scale"] is not None:
            z *= s["scale"].double()
        if s["bias"] is not None:
            z += s["bias"].double()
        z = {"none": lambda: z, "relu": lambda: z.relu(), "silu": lambda: z * z.sigmoid(),
             "swiglu": lambda: z[:, :case["N"]] * z[:, :case["N"]].sigmoid() * z[:, case["N"]:],
             "gelu": lambda: z * (0.5 * torch.erfc(-z / 2 ** 0.5)),
             "gelu_tanh": lambda: z * torch.sigmoid((8 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)),
             }[case["act"]]()
        return z if s["residual"] is None else z + s["residual"].double()

    # route: rounds of "the largest, then the lowest id" on the host
    T, E, G, k = case["T"], case["E"], case["G"], case["k"]
    lg = s["logits"].cpu().numpy().astype(np.float64)
    off = ~np.isfinite(lg)
    if s["mask"] is not None:
        off |= ~s["mask"].cpu().numpy()[:, None]
    lg = np.where(off, -np.inf, lg)
    rows = np.arange(T)
    none = off.all(1)
    peak = np.where(none, 0.0, lg.max(1))[:, None]
    soft = np.exp(lg - peak)
    score = 1.0 / (1.0 + np.exp(-np.where(off, 0.0, lg))) if case["scoring"] == "sigmoid" else \
        soft / np.where(none, 1.0, soft.sum(1))[:, None]
    if s["bias"] is not None:
        key = score + s["bias"].cpu().numpy().astype(np.float64)
    elif G > 1 and case["group_score"] == "top2":
        key = score
    else:
        key = lg
    key = np.where(off, -np.inf, key)
    if G > 1:
        parts = key.reshape(T, G, E // G)
        first = parts.max(2)
        if case["group_score"] == "top2" and E // G > 1:
            second = np.partition(parts, E // G - 2, axis=2)[:, :, E // G - 2]
            first = first + np.where(np.isinf(second), 0.0, second)
        left = first.copy()
        keep = np.zeros((T, G), bool)
        for _ in range(case["tg"]):
            at = np.argmax(np.where(keep, -np.inf, left), 1)
            taken = keep[rows, at]
            keep[rows[~taken], at[~taken]] = True
        key = np.where(np.repeat(keep, E // G, axis=1), key, -np.inf)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    src = soft if case["scoring"] == "softmax" and case["renorm"] else score
    for j in range(k):
        at = np.argmax(key, 1)
        live = key[rows, at] > -np.inf
        ids[live, j] = at[live]
        w[live, j] = src[rows[live], at[live]]
        key[rows, at] = -np.inf
    if case["renorm"]:
        total = w.sum(1)
        w /= np.where(total > 0, total, 1.0)[:, None]
    return ids, case["scale"] * w
