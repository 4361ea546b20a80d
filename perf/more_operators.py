"""The measured cases of three operators of the block around the layer: the dense projection with a
batch's adapters inside its epilogue (`linear_lora`), the norms before and after a block with its gate
and residual scales (`block_norm`), and the whole layer for a few tokens (`forward_few`).

`run` with `own` false computes them from elementary torch operations; with `own` true it calls
the library. Every case is built from its sizes and a seed alone."""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # --- linear_lora ---
        # one token of a request with its adapter, square projection onto the residual: latency
        dict(name="lora_one", op="lora", T=1, K=4096, N=4096, act="none", w="bf16", nA=8, r=16, ids="random",
             none=0.0, bias=True, residual=True, pad=0),
        # the decode batch through a shared expert's gate_up, adapters before SiLU-and-mul
        dict(name="lora_decode_gate_up", op="lora", T=64, K=4096, N=11008, act="swiglu", w="bf16", nA=8, r=16,
             ids="random", none=0.0, bias=False, residual=False, pad=0),
        # a large batch of many tenants, some tokens on the base model
        dict(name="lora_batch", op="lora", T=256, K=4096, N=4096, act="none", w="bf16", nA=64, r=16, ids="random",
             none=0.1, bias=False, residual=True, pad=0),
        # nothing divides a tile: odd rows and columns, E4M3 weights, x a slice of a wider buffer, several
        # requests' chunks of prompt one after another
        dict(name="lora_ragged_e4m3", op="lora", T=777, K=2032, N=1531, act="gelu_tanh", w="e4m3", nA=5, r=8,
             ids="runs", none=0.2, bias=True, residual=True, pad=80),
        # prompts of several tenants through a shared expert's gate_up
        dict(name="lora_prompt_gate_up", op="lora", T=4096, K=4096, N=14336, act="swiglu", w="bf16", nA=32, r=64,
             ids="runs", none=0.0, bias=False, residual=False, pad=0),
        # --- block_norm ---
        # one token between two layers: residual add and the next norm, latency only
        dict(name="norm_one", op="norm", T=1, h=4096, norm="rms", post=False, gate="none", pad=0),
        # odd rows, LayerNorm, a gate for each feature shared by the tokens, rows of wider buffers
        dict(name="norm_odd", op="norm", T=1531, h=2043, norm="layer", post=True, gate="feature", pad=7),
        # prompts: norm after the block, a gate for each token, residual add, norm before the next block
        dict(name="norm_prompt", op="norm", T=16384, h=4096, norm="rms", post=True, gate="token", pad=0),
        # --- forward_few ---
        # one token through fine-grained experts: the layer's latency
        dict(name="few_one_fine_grained", op="few", T=1, h=2048, I=768, E=128, k=8, nA=64, r=32, w="bf16",
             given=False, none=0.0, empty=0.0),
        # one token through large experts: weight streaming
        dict(name="few_one", op="few", T=1, h=4096, I=11008, E=16, k=2, nA=8, r=16, w="bf16", given=False,
             none=0.0, empty=0.0),
        # some requests at once, E4M3 experts, choices of another router with empty slots, base-model tokens
        dict(name="few_given_e4m3", op="few", T=5, h=4096, I=11008, E=16, k=2, nA=8, r=16, w="e4m3", given=True,
             none=0.3, empty=0.2),
        # the largest batch it takes, experts shared by some tokens
        dict(name="few_batch_fine_grained", op="few", T=16, h=2048, I=768, E=128, k=8, nA=64, r=32, w="bf16",
             given=False, none=0.0, empty=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST_FLOPS = 2 * 4096 * 4096 * 2 * 14336  # of the largest listed projection
_MOST_ELEMENTS = 16384 * 4096              # of the largest listed norm
_MOST_EXPERT_BYTES = 2 * 3 * 4096 * 11008 * 16


def draw(rng):
    what = rng.random()
    if what < 0.4:
        T, w = _log(rng, 1, 8192), rng.choice(["bf16", "bf16", "e4m3"])
        act = rng.choice(["none", "none", "silu", "gelu_tanh", "swiglu", "swiglu"])
        K = 16 * _log(rng, 8, 512) + (8 if w == "bf16" and rng.random() < 0.5 else 0)
        most = _MOST_FLOPS // (3 * T * K * (2 if act == "swiglu" else 1))
        return dict(op="lora", T=T, K=K, N=max(1, min(_log(rng, 64, 16384), most)), act=act, w=w, nA=_log(rng, 1, 64),
                    r=rng.choice([8, 16, 32, 64]), ids=rng.choice(["random", "runs"]) if T <= 512 else "runs",
                    none=rng.choice([0.0, 0.1, 0.5]), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8 if w == "bf16" else 16, 128]))
    if what < 0.65:
        h = _log(rng, 64, 16384)
        return dict(op="norm", T=_log(rng, 1, min(65536, _MOST_ELEMENTS // h)), h=h, norm=rng.choice(["rms", "rms", "layer"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "token", "feature", "element"]),
                    pad=rng.choice([0, 0, 8, 3]))
    E = _log(rng, 4, 128)
    k = min(E, _log(rng, 1, 8))
    h, I = 128 * _log(rng, 4, 32), 128 * _log(rng, 2, 86)
    while E * 3 * h * I * 2 > _MOST_EXPERT_BYTES:
        I = 128 * max(1, I // 256)
    nA, r = _log(rng, 1, 64), rng.choice([8, 16, 32, 64])
    while nA * E * r * (2 * h + 3 * I) * 2 > _MOST_EXPERT_BYTES:
        nA //= 2
    given = rng.random() < 0.4
    return dict(op="few", T=_log(rng, 1, 16), h=h, I=I, E=E, k=k, nA=nA, r=r, w=rng.choice(["bf16", "bf16", "e4m3"]),
                given=given, none=rng.choice([0.0, 0.2]), empty=0.2 if given and rng.random() < 0.5 else 0.0)


def _codes(W):
    """E4M3 codes with one scale per row, the largest magnitude of a row at 448."""
    scale = (W.abs().amax(-1) / 448.0).clamp_min(1e-12)
    return (W / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 6007 + 29)

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * sigma)

    def small(*shape):  # weights: in bf16, a leading index at a time
        out = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
        for part in out:
            part.copy_(0.02 * torch.randn(part.shape, generator=g, device=DEV))
        return out

    def rows(T, n, pad):  # a slice of a wider buffer
        return normal(T, n + pad).bfloat16()[:, :n]

    def adapters(T, nA, pattern, none):
        if pattern == "runs":  # one request's tokens after another's, of 64 to 512 tokens
            n = T // 64 + 2
            lengths = torch.randint(64, 513, (n,), generator=g, device=DEV)
            of = torch.searchsorted(lengths.cumsum(0), torch.arange(T, device=DEV), right=True).clamp_max(n - 1)
            ids = torch.randint(0, nA, (n,), generator=g, device=DEV)
            ids = torch.where(torch.rand(n, generator=g, device=DEV) < none, -1, ids)[of]
        else:
            ids = torch.randint(0, nA, (T,), generator=g, device=DEV)
            ids = torch.where(torch.rand(T, generator=g, device=DEV) < none, -1, ids)
        return ids.int()

    s = dict(case=case)
    T = case["T"]
    if case["op"] == "lora":
        K, N, nA, r = case["K"], case["N"], case["nA"], case["r"]
        out = 2 * N if case["act"] == "swiglu" else N
        s["x"] = rows(T, K, case["pad"])
        W = normal(out, K, sigma=0.02)
        s["W"], s["scale"] = _codes(W) if case["w"] == "e4m3" else (W.bfloat16(), None)
        s["A"], s["B"] = small(nA, r, K), small(nA, out, r)
        s["ids"] = adapters(T, nA, case["ids"], case["none"])
        s["bias"] = normal(out).bfloat16() if case["bias"] else None
        s["residual"] = normal(T, N).bfloat16() if case["residual"] else None
        return s
    if case["op"] == "norm":
        h, pad = case["h"], case["pad"]
        # a residual stream grows over the layers and has a few large features
        features = 1.0 + 10.0 * (torch.rand(h + pad, generator=g, device=DEV) < 0.01)
        s["y"] = rows(T, h, pad)
        s["residual"] = (3.0 * normal(T, h + pad) * features).bfloat16()[:, :h]
        s["weight"] = (1.0 + normal(h, sigma=0.1)).bfloat16()
        s["post"] = (1.0 + normal(h, sigma=0.1)).bfloat16() if case["post"] else None
        layer = case["norm"] == "layer"
        s["bias"] = normal(h, sigma=0.1).bfloat16() if layer else None
        s["post_bias"] = normal(h, sigma=0.1).bfloat16() if layer and case["post"] else None
        s["gate"] = {"none": lambda: None, "token": lambda: normal(T),
                     "feature": lambda: normal(1, h).bfloat16().expand(T, h),
                     "element": lambda: rows(T, h, pad)}[case["gate"]]()
        return s
    h, I, E, k, nA, r = (case[n] for n in ("h", "I", "E", "k", "nA", "r"))
    s["x"] = normal(T, h).bfloat16()
    s["W1"], s["W2"] = small(E, 2 * I, h), small(E, h, I)
    s["s1"] = s["s2"] = None
    if case["w"] == "e4m3":
        for name, scale in (("W1", "s1"), ("W2", "s2")):
            pairs = [_codes(W.float()) for W in s[name]]
            s[name], s[scale] = torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])
    s["A1"], s["B1"] = small(nA, E, r, h), small(nA, E, 2 * I, r)
    s["A2"], s["B2"] = small(nA, E, r, I), small(nA, E, h, r)
    s["ids"] = adapters(T, nA, "random", case["none"])
    logits = normal(T, E)
    if case["given"]:  # sigmoid scores of another router, some slots left empty
        best = logits.topk(k, dim=1)
        w = torch.sigmoid(best.values)
        off = torch.rand(T, k, generator=g, device=DEV) < case["empty"]
        s["topk_ids"] = torch.where(off, -1, best.indices).int()
        s["topk_w"] = torch.where(off, 0.0, w / w.sum(1, keepdim=True))
    else:
        s["logits"] = logits
    return s


def _weights(W, scale):
    return W.float() if scale is None else W.view(torch.float8_e4m3fn).float() * scale[..., None]


def _lora_plain(s, c):
    x, ids = s["x"].float(), s["ids"].long()
    v = torch.matmul(x, _weights(s["W"], s["scale"]).t())
    some = (ids >= 0)[:, None]
    if c["ids"] == "runs":  # adapter by adapter: most tokens share theirs
        for a in range(c["nA"]):
            term = torch.matmul(torch.matmul(x, s["A"][a].float().t()), s["B"][a].float().t())
            v = torch.where((ids == a)[:, None], v + term, v)
    else:
        step = 8
        for t in range(0, c["T"], step):
            a = ids[t:t + step].clamp_min(0)
            z = (x[t:t + step, None, :] * s["A"][a].float()).sum(2)
            term = (z[:, None, :] * s["B"][a].float()).sum(2)
            v[t:t + step] += torch.where(some[t:t + step], term, 0.0)
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if c["act"] == "swiglu":
        gate, up = v[:, :c["N"]], v[:, c["N"]:]
        v = gate / (1.0 + torch.exp(-gate)) * up
    elif c["act"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif c["act"] == "gelu_tanh":
        v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.bfloat16()


EPS, RESIDUAL_SCALE, BRANCH_SCALE = 1e-6, 1.0, 0.5


def _norm_plain(s, c):
    def norm(v, weight, bias):
        if c["norm"] == "layer":
            v = v - v.mean(1, keepdim=True)
        v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * weight.float()
        return v if bias is None else v + bias.float()

    b = s["y"].float()
    if s["post"] is not None:
        b = norm(b, s["post"], s["post_bias"])
    if c["gate"] == "token":
        b = b / (1.0 + torch.exp(-s["gate"]))[:, None]
    elif s["gate"] is not None:
        b = b * s["gate"].float()
    total = RESIDUAL_SCALE * s["residual"].float() + BRANCH_SCALE * b
    return total.bfloat16(), norm(total, s["weight"], s["bias"]).bfloat16()


def _few_plain(s, c):
    T, k, I = c["T"], c["k"], c["I"]
    if c["given"]:
        ids, w = s["topk_ids"].long(), s["topk_w"]
    else:
        best, ids = s["logits"].sort(dim=1, descending=True, stable=True)
        best, ids = best[:, :k], ids[:, :k]
        w = torch.exp(best - best[:, :1])
        w = w / w.sum(1, keepdim=True)
    x, out = s["x"].float(), []
    for t in range(T):
        total = torch.zeros(c["h"], device=DEV)
        a = s["ids"][t:t + 1].long()
        for j in range(k):
            e = ids[t, j:j + 1]
            at, of = e.clamp_min(0), a.clamp_min(0)

            def term(v, W, scale, A, B):
                base = torch.matmul(_weights(W.index_select(0, at)[0], None if scale is None else scale.index_select(0, at)[0]), v)
                z = torch.matmul(A.index_select(0, of)[0].index_select(0, at)[0].float(), v)
                more = torch.matmul(B.index_select(0, of)[0].index_select(0, at)[0].float(), z)
                return base + torch.where(a >= 0, more, 0.0)

            v = term(x[t], s["W1"], s["s1"], s["A1"], s["B1"])
            act = v[:I] / (1.0 + torch.exp(-v[:I])) * v[I:]
            v = term(act, s["W2"], s["s2"], s["A2"], s["B2"])
            total = total + torch.where(e >= 0, w[t, j] * v, 0.0)
        out.append(total)
    return torch.stack(out).bfloat16()


def run(state):
    c, s = state["case"], state
    if not own:
        return {"lora": _lora_plain, "norm": _norm_plain, "few": _few_plain}[c["op"]](s, c)
    import lora_mixture_experts_amd as ml

    if c["op"] == "lora":
        return ml.linear_lora(s["x"], s["W"], s["A"], s["B"], s["ids"], w_scale=s["scale"], bias=s["bias"],
                              act=c["act"], residual=s["residual"])
    if c["op"] == "norm":
        return ml.block_norm(s["y"], s["residual"], s["weight"], bias=s["bias"], post_weight=s["post"],
                             post_bias=s["post_bias"], gate=s["gate"], sigmoid_gate=c["gate"] == "token",
                             residual_scale=RESIDUAL_SCALE, branch_scale=BRANCH_SCALE, norm=c["norm"], eps=EPS)
    if c["given"]:
        return ml.forward_few(s["x"], s["W1"], s["W2"], s["A1"], s["B1"], s["A2"], s["B2"], s["ids"],
                              topk_ids=s["topk_ids"], topk_w=s["topk_w"], W1_scale=s["s1"], W2_scale=s["s2"])
    return ml.forward_few(s["x"], s["W1"], s["W2"], s["A1"], s["B1"], s["A2"], s["B2"], s["ids"],
                          router_logits=s["logits"], topk=c["k"], W1_scale=s["s1"], W2_scale=s["s2"])


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        h = case["h"]
        nbytes = 8 * T * h + 2 * h * (1 + int(case["post"])) * (2 if case["norm"] == "layer" else 1)
        nbytes += {"none": 0, "token": 4 * T, "feature": 2 * h, "element": 2 * T * h}[case["gate"]]
        return dict(bytes=nbytes, flops=T * h * (14 if case["post"] else 8))
    nA, r = case["nA"], case["r"]
    with_adapter = T * (1.0 - case["none"])
    if case["op"] == "lora":
        K, N = case["K"], case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        # requests of a prompt have some 288 tokens each; a batch's tokens choose alike among the adapters
        picks = with_adapter / 288 + 1 if case["ids"] == "runs" and T > 288 else \
            1 if case["ids"] == "runs" else with_adapter
        used = nA * (1.0 - (1.0 - 1.0 / nA) ** picks)
        nbytes = 2 * T * K + (rows * (K + 4) if case["w"] == "e4m3" else 2 * rows * K) + 2 * T * N + 4 * T
        nbytes += 2 * used * r * (K + rows)
        nbytes += (2 * rows if case["bias"] else 0) + (2 * T * N if case["residual"] else 0)
        return dict(bytes=int(nbytes), flops=int(2 * T * K * rows + 2 * with_adapter * r * (K + rows)))
    h, I, E, k = case["h"], case["I"], case["E"], case["k"]
    slots = k * (1.0 - case["empty"])
    experts = E * (1.0 - (1.0 - slots / E) ** T)
    pairs, carrying = T * slots, with_adapter * slots
    used = nA * E * (1.0 - (1.0 - 1.0 / (nA * E)) ** carrying)
    nbytes = experts * ((3 * h * I + 4 * (2 * I + h)) if case["w"] == "e4m3" else 6 * h * I)
    nbytes += used * 2 * r * (2 * h + 3 * I) + 4 * T * h + 4 * T
    nbytes += 8 * T * k if case["given"] else 4 * T * E
    return dict(bytes=int(nbytes), flops=int(2 * pairs * 3 * h * I + 2 * carrying * r * (2 * h + 3 * I)))


def exact(case, seed):
    s, c, T = prepare(case, seed), case, case["T"]

    def decoded(W, scale):
        return W.double() if scale is None else W.view(torch.float8_e4m3fn).double() * scale.double().unsqueeze(-1)

    if c["op"] == "norm":
        def norm(v, w, b):
            centre = v.mean(1, keepdim=True) if c["norm"] == "layer" else 0.0
            v = v - centre
            v = v * (v.square().sum(1, keepdim=True) / c["h"] + EPS).rsqrt() * w.double()
            return v if b is None else v + b.double()

        b = s["y"].double()
        b = b if s["post"] is None else norm(b, s["post"], s["post_bias"])
        if s["gate"] is not None:
            b = b * (torch.sigmoid(s["gate"].double()).unsqueeze(1) if c["gate"] == "token" else s["gate"].double())
        total = s["residual"].double() * RESIDUAL_SCALE + b * BRANCH_SCALE
        return total, norm(total, s["weight"], s["bias"])

    if c["op"] == "lora":
        v = s["x"].double() @ decoded(s["W"], None).T if s["scale"] is None else \
            (s["x"].double() @ s["W"].view(torch.float8_e4m3fn).double().T) * s["scale"].double()
        ids = s["ids"].tolist()
        for a in sorted(set(ids) - {-1}):
            rows = torch.tensor([t for t in range(T) if ids[t] == a], device=DEV)
            v[rows] += (s["x"][rows].double() @ s["A"][a].double().T) @ s["B"][a].double().T
        if s["bias"] is not None:
            v += s["bias"].double()
        if c["act"] == "swiglu":
            v = torch.sigmoid(v[:, :c["N"]]) * v[:, :c["N"]] * v[:, c["N"]:]
        elif c["act"] == "silu":
            v = v * torch.sigmoid(v)
        elif c["act"] == "gelu_tanh":
            v = v * torch.sigmoid((8 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
        return v if s["residual"] is None else v + s["residual"].double()

    # few: expert by expert over the tokens that chose it
    E, k, I = c["E"], c["k"], c["I"]
    chosen = []  # (expert, token, weight)
    if c["given"]:
        ids, w = s["topk_ids"].tolist(), s["topk_w"].double().tolist()
        chosen = [(ids[t][j], t, w[t][j]) for t in range(T) for j in range(k) if ids[t][j] >= 0]
    else:
        for t, row in enumerate(s["logits"].tolist()):
            best = sorted(range(E), key=lambda e: (-row[e], e))[:k]
            u = [math.exp(row[e] - row[best[0]]) for e in best]
            chosen += [(e, t, v / math.fsum(u)) for e, v in zip(best, u)]
    x, ad = s["x"].double(), s["ids"].tolist()
    y = torch.zeros(T, c["h"], dtype=torch.float64, device=DEV)
    for e in sorted({p[0] for p in chosen}):
        W1 = decoded(s["W1"][e], None if s["s1"] is None else s["s1"][e])
        W2 = decoded(s["W2"][e], None if s["s2"] is None else s["s2"][e])
        for _, t, w in [p for p in chosen if p[0] == e]:
            v = W1 @ x[t]
            if ad[t] >= 0:
                v += s["B1"][ad[t], e].double() @ (s["A1"][ad[t], e].double() @ x[t])
            act = v[:I] * torch.sigmoid(v[:I]) * v[I:]
            out = W2 @ act
            if ad[t] >= 0:
                out += s["B2"][ad[t], e].double() @ (s["A2"][ad[t], e].double() @ act)
            y[t] += w * out
    return y
