"""The layer for a few tokens (moe_lora_forward_few) against float64. The bound per element carries the fp32
errors (n additions of at most 2^-24 of the sum of magnitudes for a sum of n terms; 2^-20 for the
exponentials, reciprocals and the softmax) and the activations' two bf16 (2^-8 of 2^-8) through the formulas,
and half a bf16 step of the result."""
import ctypes
import math
import threading

import pytest
import torch

import lora_mixture_experts_amd as ml
from tests.test_block_norm import _reference as norm_reference
from tests.test_block_norm import _within
from tests.test_linear_lora import _compare as compare_lora

DEV = "cuda"
BF = torch.bfloat16
U = 2.0 ** -24


def _make(T, h, I, E, k, nA, r, w="bf16", seed=0, none=0.25):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1000 * T + h + I + E)

    def normal(*shape, sigma=1.0):
        return sigma * torch.randn(*shape, generator=g, device=DEV)

    s = dict(x=normal(T, h).to(BF), W1=normal(E, 2 * I, h, sigma=h ** -0.5), W2=normal(E, h, I, sigma=I ** -0.5),
             A1=normal(nA, E, r, h, sigma=h ** -0.5).to(BF), B1=normal(nA, E, 2 * I, r, sigma=0.5).to(BF),
             A2=normal(nA, E, r, I, sigma=I ** -0.5).to(BF), B2=normal(nA, E, h, r, sigma=0.5).to(BF))
    s["W1_scale"] = s["W2_scale"] = None
    for n in ("W1", "W2"):
        if w == "e4m3":
            scale = (s[n].abs().amax(-1) / 448).clamp_min(1e-20)
            s[n], s[n + "_scale"] = (s[n] / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale
        else:
            s[n] = s[n].to(BF)
    ids = torch.randint(0, nA, (T,), generator=g, device=DEV)
    s["adapter_ids"] = torch.where(torch.rand(T, generator=g, device=DEV) < none, -1, ids).int()
    logits = normal(T, E)
    return s, logits


def _choice(logits, k):
    best, ids = logits.double().sort(dim=1, descending=True, stable=True)
    return ids[:, :k].int(), torch.softmax(best[:, :k], 1)


def _decode(W, scale):
    return W.double() if scale is None else W.view(torch.float8_e4m3fn).double() * scale.double()[:, None]


def _reference(s, ids, w):
    """(y, bound) in float64: every pair written out."""
    x, ad = s["x"].double(), s["adapter_ids"].tolist()
    T, h = x.shape
    E, I, r, nA = s["W1"].shape[0], s["W2"].shape[2], s["A1"].shape[2], s["A1"].shape[0]
    y, dy = torch.zeros(T, h, dtype=torch.float64, device=DEV), torch.zeros(T, h, dtype=torch.float64, device=DEV)
    idl, wl = ids.tolist(), w.double().tolist()
    cache = {}

    def project(v, dv, W, A, B):
        out, n = W @ v, v.numel()
        d = W.abs() @ dv + (n + 4) * U * (W.abs() @ v.abs()) + 4 * U * out.abs()
        if A is not None:
            z = A @ v
            dz = A.abs() @ dv + (n + 4) * U * (A.abs() @ v.abs())
            more = B @ z
            d = d + B.abs() @ dz + (r + 2) * U * (B.abs() @ z.abs())
            out = out + more
        return out, d + U * out.abs()

    for t in range(T):
        for j, e in enumerate(idl[t]):
            if not 0 <= e < E:
                continue
            if e not in cache:
                cache.clear()
                cache[e] = [_decode(s[n][e], None if s[n + "_scale"] is None else s[n + "_scale"][e]) for n in ("W1", "W2")]
            W1, W2 = cache[e]
            a = ad[t] if 0 <= ad[t] < nA else None
            lora = [None if a is None else s[n][a, e].double() for n in ("A1", "B1", "A2", "B2")]
            v, dv = project(x[t], torch.zeros_like(x[t]), W1, lora[0], lora[1])
            g, u, dg, du = v[:I], v[I:], dv[:I], dv[I:]
            act = g * torch.sigmoid(g) * u
            dact = 1.1 * dg * (u.abs() + du) + g.abs() * du + (2.0 ** -20 + 2.0 ** -16) * act.abs()
            out, dout = project(act, dact, W2, lora[2], lora[3])
            wt = wl[t][j]
            y[t] += wt * out
            dy[t] += abs(wt) * (dout + 2.0 ** -20 * out.abs())
    dy = dy + (len(idl[0]) + 10) * U * y.abs()
    return y, dy + 2.0 ** -8 * (y.abs() + dy) + 2.0 ** -126


def _compare(y, ref):
    assert torch.isfinite(y).all()
    worst = ((y.double() - ref[0]).abs() / ref[1]).max().item()
    assert worst <= 1.0, worst


SHAPES = [
    # T, h, I, E, k, adapters, rank
    (1, 128, 128, 1, 1, 1, 8), (1, 256, 384, 8, 2, 3, 16), (1, 1024, 768, 128, 8, 4, 32), (2, 384, 256, 5, 5, 2, 64),
    (3, 2048, 128, 16, 2, 7, 16), (5, 128, 1408, 6, 3, 9, 8), (7, 640, 640, 300, 4, 2, 32), (8, 256, 512, 8, 8, 8, 16),
    (13, 512, 384, 17, 16, 3, 8), (16, 256, 256, 32, 8, 16, 32), (16, 1152, 896, 4, 2, 5, 64), (16, 128, 128, 1024, 16, 2, 16),
    (16, 4096, 2048, 16, 2, 2, 16),
    # every token on the same experts, mostly with adapters of their own
    (16, 128, 128, 1, 1, 1, 8), (16, 4096, 256, 1, 1, 40, 16), (15, 2048, 384, 2, 2, 33, 64), (9, 4096, 11008, 1, 1, 16, 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_few_matches_float64(shape, w):
    print("forward_few", shape, w, flush=True)
    T, h, I, E, k, nA, r = shape
    s, logits = _make(*shape, w)
    y = ml.forward_few(**s, router_logits=logits, topk=k)
    torch.cuda.synchronize()
    _compare(y, _reference(s, *_choice(logits, k)))
    assert torch.equal(y, ml.forward_few(**s, router_logits=logits, topk=k)), "not the same bits twice"


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_few_routes_as_the_layer(shape):
    """From the logits, with ties among them, as from the layer's own choice; and the layer's result up to
    its rounding of the activations."""
    T, h, I, E, k, nA, r = shape
    s, logits = _make(*shape, seed=3)
    logits = (logits * 2).round() / 2
    d = ml.dims_of(s["x"], s["W1"], s["A1"])
    own = ml.route_align(logits, s["adapter_ids"], k, d)
    y = ml.forward_few(**s, router_logits=logits, topk=k)
    assert torch.equal(y, ml.forward_few(**s, topk_ids=own["topk_ids"], topk_w=own["topk_w"]))
    order = [s[n] for n in ("W1", "W2", "A1", "B1", "A2", "B2")]
    layer = ml.forward(s["x"], logits, *order, s["adapter_ids"], k).double()
    assert (y.double() - layer).abs().max() <= 2e-2 * layer.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 16])
@pytest.mark.parametrize("empty", [0.0, 0.4, 0.95])
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_few_empty_slots_and_repeated_experts(T, empty, w):
    h, I, E, k, nA, r = 256, 384, 6, 5, 3, 16
    s, _ = _make(T, h, I, E, k, nA, r, w, seed=7)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E, (T, k), generator=g)  # experts named twice among them
    off = torch.rand(T, k, generator=g) < empty
    wt = torch.rand(T, k, generator=g) - 0.25
    wt[off] = math.nan  # the weight of an empty slot is not used
    ids = torch.where(off, -1, ids).int().to(DEV)
    y = ml.forward_few(**s, topk_ids=ids, topk_w=wt.to(DEV))
    _compare(y, _reference(s, ids, torch.where(off, 0.0, wt)))
    none = ml.forward_few(**s, topk_ids=torch.full_like(ids, -1), topk_w=wt.to(DEV))
    assert (none == 0).all()


@pytest.mark.gpu
def test_few_flags():
    """Logits that are not finite count as -infinity; ids out of range as none. The flags tell."""
    T, h, I, E, k, nA, r = 5, 256, 256, 8, 3, 2, 8
    s, logits = _make(T, h, I, E, k, nA, r, seed=9)
    ws = torch.full((4 << 20,), 255, dtype=torch.uint8, device=DEV)
    want = ml.forward_few(**s, router_logits=logits, topk=k, workspace=ws)
    assert ml.debug_status(ws) == 0
    bad = logits.clone()
    bad[2, 1], bad[2, 4] = math.nan, math.inf
    low = logits.clone()
    low[2, 1], low[2, 4] = -3e38, -3.1e38
    y = ml.forward_few(**s, router_logits=bad, topk=k, workspace=ws)
    assert ml.debug_status(ws) == ml.FLAG_NONFINITE_LOGIT
    assert torch.equal(y, ml.forward_few(**s, router_logits=low, topk=k))
    ids, w = _choice(logits, k)
    w = w.float()
    a = s["adapter_ids"].clone()
    a[0], a[1] = nA, -5
    fine = s["adapter_ids"].clone()
    fine[0], fine[1] = -1, -1
    y = ml.forward_few(**{**s, "adapter_ids": a}, topk_ids=ids, topk_w=w, workspace=ws)
    assert ml.debug_status(ws) == ml.FLAG_ADAPTER_RANGE
    assert torch.equal(y, ml.forward_few(**{**s, "adapter_ids": fine}, topk_ids=ids, topk_w=w))
    far, near = ids.clone(), ids.clone()
    far[3, 0], far[4, 2] = E, -7
    near[3, 0], near[4, 2] = -1, -1
    y = ml.forward_few(**s, topk_ids=far, topk_w=w, workspace=ws)
    assert ml.debug_status(ws) == ml.FLAG_EXPERT_RANGE
    assert torch.equal(y, ml.forward_few(**s, topk_ids=near, topk_w=w))
    assert torch.isfinite(want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_few_broken_weights_stay_with_their_tokens(bad):
    """Infinities and NaNs of one expert, of one adapter and of one token reach nobody else."""
    T, h, I, E, k, nA, r = 12, 256, 384, 8, 2, 4, 16
    s, logits = _make(T, h, I, E, k, nA, r, seed=11)
    ids, w = _choice(logits, k)
    w = w.float()
    want = ml.forward_few(**s, topk_ids=ids, topk_w=w)
    has = {e: (ids == e).any(1) for e in range(E)}
    for name in ("W1", "W2"):
        t = s[name].clone()
        t[3, 5, 7] = bad
        y = ml.forward_few(**{**s, name: t}, topk_ids=ids, topk_w=w)
        assert torch.equal(y[~has[3]], want[~has[3]])
        assert not torch.isfinite(y[has[3]]).all(1).any()
    for name in ("A1", "B1", "A2", "B2"):
        t = s[name].clone()
        t[2, :, 1, 3] = bad
        y = ml.forward_few(**{**s, name: t}, topk_ids=ids, topk_w=w)
        others = s["adapter_ids"] != 2
        assert torch.equal(y[others], want[others])
        assert not torch.isfinite(y[~others]).all(1).any()
    x = s["x"].clone()
    x[4, 9] = bad
    y = ml.forward_few(**{**s, "x": x}, topk_ids=ids, topk_w=w)
    rows = [t for t in range(T) if t != 4]
    assert torch.equal(y[rows], want[rows]) and not torch.isfinite(y[4]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 512, 768, 16, 4, 3, 16), (16, 256, 256, 32, 8, 16, 32)], ids=str)
def test_few_poisoned_workspace_and_other_streams(shape):
    T, h, I, E, k, nA, r = shape
    s, logits = _make(*shape, seed=13)
    want = ml.forward_few(**s, router_logits=logits, topk=k)
    d = ml.dims_of(s["x"], s["W1"], s["A1"])
    need = ml.lib().moe_lora_few_workspace_size(ctypes.byref(d), k)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = ml.forward_few(**s, router_logits=logits, topk=k, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert (ws[need:] == 255).all()


@pytest.mark.gpu
def test_few_experts_and_adapters_past_4_gib():
    """Byte offsets of the last expert's weights and of the last adapter's past 32 bits."""
    h, I, E, k, nA, r = 4096, 4096, 48, 2, 600, 64
    shape = dict(W1=(E, 2 * I, h), W2=(E, h, I), A1=(nA, E, r, h), B1=(nA, E, 2 * I, r))
    few, _ = _make(3, h, I, 1, 1, 1, r, none=0.0)
    s = {n: torch.zeros(shape[n], dtype=BF, device=DEV) for n in ("W1", "W2")}  # 3.2 and 1.6 GB
    big = torch.zeros(nA, E, r, h, dtype=BF, device=DEV)  # 15 GB, also as A2
    b1 = torch.zeros(nA, E, 2 * I, r, dtype=BF, device=DEV)
    s.update(A1=big, B1=b1, A2=torch.zeros(nA, E, r, I, dtype=BF, device=DEV),
             B2=torch.zeros(nA, E, h, r, dtype=BF, device=DEV))
    for n in ("W1", "W2"):
        s[n][-1] = few[n][0]
    for n in ("A1", "B1", "A2", "B2"):
        s[n][-1, -1] = few[n][0, 0]
    ids = torch.tensor([[E - 1, 0], [1, E - 1], [2, 3]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.75, 0.25]] * 3, device=DEV)
    ad = torch.tensor([nA - 1, -1, nA - 1], dtype=torch.int32, device=DEV)
    y = ml.forward_few(few["x"], **s, adapter_ids=ad, topk_ids=ids, topk_w=w)
    one = {**few, "adapter_ids": torch.tensor([0, -1, -1], dtype=torch.int32, device=DEV)}
    own = torch.tensor([[0, -1], [-1, 0], [-1, -1]], dtype=torch.int32, device=DEV)
    _compare(y, _reference(one, own, w))


@pytest.mark.gpu
def test_few_from_two_threads():
    cases = []
    for shape in ((1, 512, 768, 16, 4, 3, 16), (9, 384, 256, 12, 3, 4, 8), (16, 256, 256, 32, 8, 16, 32)):
        s, logits = _make(*shape, seed=17)
        cases.append((s, logits, shape[4]))

    def calls():
        return [ml.forward_few(**s, router_logits=logits, topk=k) for s, logits, k in cases]

    want = calls()
    torch.cuda.synchronize()
    right = []

    def work():
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(100):
                got = calls()
                side.synchronize()
                right.append(all(torch.equal(g, v) for g, v in zip(got, want)))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(right) == 200 and all(right)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12])
def test_a_decode_block_eager_and_captured(T):
    """The operators as a decode step of one block runs them: the residual stream and the norm, a projection
    with the tokens' adapters, the sum and the norm, router logits, choice, the layer for a few tokens, the
    gated sum after its norm. Each step against float64 on its own inputs; then the run captured and replayed
    on other inputs, against the eager run."""
    h, I, E, k, nA, r = 512, 384, 16, 3, 4, 16
    s, _ = _make(T, h, I, E, k, nA, r, seed=19)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)

    def normal(*shape, sigma=1.0):
        return (sigma * torch.randn(*shape, generator=g, device=DEV)).to(BF)

    y0, stream, Wo = normal(T, h), normal(T, h, sigma=2.0), normal(h, h, sigma=h ** -0.5)
    A, B, Wr = normal(nA, r, h, sigma=h ** -0.5), normal(nA, h, r), normal(E, h, sigma=2 * h ** -0.5)
    n1, n2, n3 = 1 + normal(h, sigma=0.1), 1 + normal(h, sigma=0.1), 1 + normal(h, sigma=0.1)
    gate = torch.randn(T, generator=g, device=DEV)
    ad = s.pop("adapter_ids")
    s.pop("x")
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=DEV)

    def block():
        res, x = ml.block_norm(y0, stream, n1)
        o = ml.linear_lora(x, Wo, A, B, ad, workspace=ws)
        res2, x2 = ml.block_norm(o, res, n2)
        logits = ml.router_logits(x2, Wr)
        ids, w = ml.route(logits, k, scoring="sigmoid", scale=1.5)
        moe = ml.forward_few(x2, **s, adapter_ids=ad, topk_ids=ids, topk_w=w, workspace=ws)
        last, _ = ml.block_norm(moe, res2, post_weight=n3, gate=gate, sigmoid_gate=True)
        return dict(res=res, x=x, o=o, res2=res2, x2=x2, ids=ids, w=w, moe=moe, last=last)

    v = block()
    torch.cuda.synchronize()
    pair = norm_reference(y0, stream, n1, None, None, None, None, False, 1.0, 1.0, "rms", 1e-6)
    _within(v["res"], pair[0])
    _within(v["x"], pair[1])
    compare_lora(v["o"], v["x"], Wo, None, None, "none", None, A, B, ad)
    pair = norm_reference(v["o"], v["res"], n2, None, None, None, None, False, 1.0, 1.0, "rms", 1e-6)
    _within(v["res2"], pair[0])
    _within(v["x2"], pair[1])
    _compare(v["moe"], _reference({**s, "x": v["x2"], "adapter_ids": ad}, v["ids"], v["w"]))
    _within(v["last"], norm_reference(v["moe"], v["res2"], None, None, n3, None, gate, True, 1.0, 1.0, "rms", 1e-6)[0])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block()
    for i in range(4):
        y0.copy_(torch.randn(T, h, device=DEV))
        ad.copy_(torch.randint(-1, nA, (T,), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in held.items()}
        want = block()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


@pytest.mark.gpu
def test_few_empty_batch():
    s, logits = _make(1, 128, 128, 2, 1, 1, 8)
    s["x"], s["adapter_ids"] = s["x"][:0], s["adapter_ids"][:0]
    assert ml.forward_few(**s, router_logits=logits[:0], topk=1).shape == (0, 128)


@pytest.mark.gpu
def test_few_refuses_tensors():
    T, h, I, E, k, nA, r = 3, 256, 128, 4, 2, 2, 8
    s, logits = _make(T, h, I, E, k, nA, r)
    ids, w = _choice(logits, k)
    w = w.float()
    good = dict(router_logits=logits, topk=k)
    for name, bad in [("W1", s["W1"][:, :2]), ("W1", s["W1"].float()), ("W2", s["W2"].transpose(1, 2)), ("A1", s["A1"][:1]),
                      ("B1", s["B1"][..., :4]), ("A2", None), ("B2", s["B2"].cpu()), ("adapter_ids", s["adapter_ids"].long()),
                      ("x", s["x"].float()), ("W1_scale", torch.zeros(E, 2 * I, device=DEV))]:
        with pytest.raises((TypeError, ValueError)):
            ml.forward_few(**{**s, name: bad}, **good)
    for call in (dict(), dict(router_logits=logits, topk=k, topk_ids=ids, topk_w=w), dict(topk_ids=ids), dict(topk_w=w),
                 dict(topk_ids=ids, topk_w=w, topk=k + 1), dict(router_logits=logits[:, :2], topk=k),
                 dict(router_logits=logits), dict(topk_ids=ids.long(), topk_w=w), dict(topk_ids=ids, topk_w=w.double())):
        with pytest.raises((TypeError, ValueError)):
            ml.forward_few(**s, **call)
    for topk in (0, E + 1, -1):
        with pytest.raises(ml.MoeLoraError):
            ml.forward_few(**s, router_logits=logits, topk=topk)
    with pytest.raises(ValueError):
        ml.forward_few(**s, **good, y=s["x"])
    with pytest.raises(ValueError):
        ml.forward_few(**s, **good, workspace=s["W1"].view(-1).view(torch.uint8))
    with pytest.raises(ml.MoeLoraError):
        ml.forward_few(**s, **good, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    many, l17 = _make(17, h, I, E, k, nA, r)
    with pytest.raises(ml.MoeLoraError):
        ml.forward_few(**many, router_logits=l17, topk=k)


def test_few_host_checks():
    lib = ml.lib()
    good = ml.Dims(4, 256, 384, 8, 3, 16)
    need = lib.moe_lora_few_workspace_size(ctypes.byref(good), 2)
    assert need > 0 and need % 256 == 0
    p = [0x10000 * (i + 1) for i in range(16)]
    names = ("x", "logits", "ids", "w", "W1", "s1", "W2", "s2", "A1", "B1", "A2", "B2", "adapters")

    def call(d=good, topk=2, ws=need, **change):
        q = dict(zip(names, p), ids=None, w=None, s1=None, s2=None, y=p[13], work=p[14])
        q.update(change)
        return lib.moe_lora_forward_few(*[q[n] for n in names], topk, ctypes.byref(d) if d else None, q["y"], q["work"], ws,
                                        None)

    for n in ("x", "logits", "W1", "W2", "A1", "B1", "A2", "B2", "adapters", "y", "work"):
        assert call(**{n: None}) == ml.ENULL, n
    for n in ("x", "W1", "W2", "A1", "B1", "A2", "B2", "y"):
        assert call(**{n: p[0] + 8}) == ml.EALIGN, n
    assert call(logits=p[1] + 2) == ml.EALIGN and call(adapters=p[1] + 1) == ml.EALIGN
    assert call(ids=p[2]) == ml.EUNSUPPORTED and call(ids=p[2], w=p[3]) == ml.EUNSUPPORTED
    assert call(logits=None, ids=p[2]) == ml.ENULL and call(s1=p[5]) == ml.ENULL and call(s2=p[5]) == ml.ENULL
    assert call(ws=need - 1) == ml.EWORKSPACE and call(work=p[14] + 16) == ml.EWORKSPACE
    assert call(None) == ml.ENULL and call(topk=0) == ml.EINVAL_DIMS and call(topk=9) == ml.EINVAL_DIMS
    for field, v in (("T", 17), ("T", -1), ("hidden", 200), ("hidden", 0), ("inter", 64), ("n_experts", 0), ("n_experts", 1025),
                     ("n_adapters", 0), ("rank", 24), ("inter", 1 << 30), ("hidden", 1 << 30)):
        d = ml.Dims.from_buffer_copy(good)
        setattr(d, field, v)
        assert call(d) == ml.EINVAL_DIMS, field
        assert lib.moe_lora_few_workspace_size(ctypes.byref(d), 2) == 0
    empty = ml.Dims(0, 256, 384, 8, 3, 16)
    assert call(empty, **{n: None for n in (*names, "y", "work")}) == ml.OK


def _infinite(shape, name):
    """Infinities of both signs in one expert's or one adapter's weights: the formula's results, with their signs."""
    T, h, I, E, k, nA, r = shape
    s, logits = _make(*shape, seed=23, none=0.0)
    ids, w = _choice(logits, k)
    w = w.float()
    ids[0, 0], s["adapter_ids"][0] = 1, 0
    t = s[name] = s[name].clone()
    t = t[1] if name[0] == "W" else t[0, 1]
    t[5, 7], t[3, 2], t[6, 0], t[6, 1] = math.inf, -math.inf, math.inf, -math.inf
    y = ml.forward_few(**s, topk_ids=ids, topk_w=w)
    ref, bound = _reference(s, ids, w)
    fin = torch.isfinite(ref)
    got, want = y.double()[~fin], ref[~fin]
    assert got.numel() and ((got == want) | (torch.isnan(got) & torch.isnan(want))).all()
    assert torch.isfinite(y[fin]).all() and ((y.double() - ref).abs() <= bound)[fin].all()
    return s, ids, w, fin, want


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 256, 384, 4, 2, 2, 16), (12, 256, 384, 4, 2, 4, 16), (16, 384, 128, 2, 2, 3, 8),
                                   (6, 4096, 256, 4, 2, 3, 32), (16, 4096, 128, 2, 1, 2, 16)], ids=str)
@pytest.mark.parametrize("name", ["W1", "W2", "A1", "B1", "A2"])
def test_few_infinite_weights(shape, name):
    """8 and 16 features a workgroup, experts of one token and of many; for W2 the layer's results too."""
    s, ids, w, fin, want = _infinite(shape, name)
    if name == "W2":
        order = [s[n] for n in ("W1", "W2", "A1", "B1", "A2", "B2")]
        layer = ml.forward_topk(s["x"], ids, w, *order, s["adapter_ids"])[~fin].double()
        assert ((layer == want) | (torch.isnan(layer) & torch.isnan(want))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 256, 384, 4, 2, 2, 8), (1, 2048, 1408, 2, 1, 3, 32), (12, 256, 384, 4, 2, 4, 16),
                                   (16, 384, 128, 2, 2, 3, 8), (16, 128, 128, 8, 8, 2, 64), (6, 4096, 256, 4, 2, 3, 32),
                                   (3, 4096, 640, 2, 2, 2, 64), (16, 4096, 128, 2, 1, 2, 16)], ids=str)
def test_few_infinite_second_expand(shape):
    """z2 of few pairs comes in parts that several lane groups take: their sum meets an infinity of B2, not they."""
    _infinite(shape, "B2")


def _col_tiles(shape):
    """Column tiles of a workgroup of the first product, from the size of the workspace that z2's parts take."""
    T, h, I, E, k, nA, r = shape
    need = ml.lib().moe_lora_few_workspace_size(ctypes.byref(ml.Dims(T, h, I, E, nA, r)), k)
    P = T * k

    def size(ct, splits):
        parts = [4 * P] * 4 + [64 * P] * 2 + [4 * P * r * splits, 4 * P * I, 4 * P * r * (I // (16 * ct))]
        return 256 + sum((n + 255) // 256 * 256 for n in parts)

    return {ct for ct in (1, 2, 4) for splits in (1, 2, 4) if size(ct, splits) == need}


FOUR_TILES = [  # some tokens an expert, all of them, one; 8 and 16 features a workgroup of the second product
    (16, 128, 256, 128, 8, 3, 8), (16, 256, 256, 128, 8, 5, 32), (13, 128, 256, 128, 16, 2, 64), (16, 256, 4096, 8, 2, 5, 32),
    (16, 128, 32768, 1, 1, 20, 64), (16, 128, 32768, 1, 1, 3, 8), (16, 4096, 1024, 32, 4, 2, 64), (3, 4096, 11008, 3, 2, 2, 8)]


def test_few_shapes_of_four_column_tiles():
    for shape in FOUR_TILES:
        assert _col_tiles(shape) == {4}, shape
    assert _col_tiles((1, 1024, 768, 128, 8, 4, 32)) == {2} and _col_tiles((2, 384, 256, 5, 5, 2, 64)) == {1}


@pytest.mark.gpu
@pytest.mark.parametrize("shape", FOUR_TILES, ids=str)
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_few_four_column_tiles(shape, w):
    """The first product's widest form at every rank, with experts of many tokens."""
    print("forward_few", shape, w, flush=True)
    s, logits = _make(*shape, w, seed=29)
    y = ml.forward_few(**s, router_logits=logits, topk=shape[4])
    _compare(y, _reference(s, *_choice(logits, shape[4])))
