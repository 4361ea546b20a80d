"""The layer from given experts and weights (moe_lora_forward_topk): bit for bit the layer's own
result on the layer's own routing, the oracle's with empty slots, repeated experts and padded rows,
and the run of operators it belongs to (router logits, route, layer, shared expert)."""
import ctypes

import numpy as np
import pytest
import torch

import lora_mixture_experts_amd as ml
import oracle
from synth import configs
from synth.configs import Workload
from tests.helpers import check_close

DEV = "cuda"
BF = torch.bfloat16

SHAPES = {
    "decode": Workload("decode_small", 37, 384, 640, 6, 2, 5, 16),
    "one_token": Workload("one_token", 1, 256, 384, 8, 2, 4, 16),
    "fine": Workload("fine", 64, 256, 256, 32, 8, 16, 32),
    "tiled64": Workload("tiled64", 256, 384, 640, 4, 2, 5, 16),
    "tiled128": Workload("tiled128", 900, 256, 384, 3, 2, 6, 64),
    "tiled192": Workload("tiled192", 500, 256, 256, 8, 2, 9, 16),
    "tiled256": Workload("tiled256", 1700, 256, 256, 2, 1, 4, 8),
    "lists_in_memory": Workload("lists", 2600, 128, 128, 16, 4, 7, 8),
}


def _gpu(inp):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in inp.items()}


def _weights(g):
    return [g[k] for k in ("W1", "W2", "A1", "B1", "A2", "B2")]


def _reference(inp, ids, w):
    """sum_j w[t][j] * expert ids[t][j], float64, each slot through the oracle's layer with one
    expert per token; empty slots and their weights left out."""
    T, k = ids.shape
    E = inp["W1"].shape[0]
    y = np.zeros((T, inp["x"].shape[1]))
    for j in range(k):
        rows = np.nonzero(ids[:, j] >= 0)[0]
        if rows.size == 0:
            continue
        sub = dict(inp)
        sub["x"] = inp["x"][torch.from_numpy(rows)]
        sub["adapter_ids"] = inp["adapter_ids"][torch.from_numpy(rows)]
        logits = torch.full((rows.size, E), -5.0)
        logits[torch.arange(rows.size), torch.from_numpy(ids[rows, j].astype(np.int64))] = 5.0
        sub["logits"] = logits
        y[rows] += w[rows, j].astype(np.float64)[:, None] * oracle.forward(sub, 1)
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHAPES)
def test_equals_the_layer_on_its_own_routing(name):
    w = SHAPES[name]
    print("forward_topk equals", name, flush=True)
    g = _gpu(configs.make_inputs(w, 1))
    d = ml.dims_of(g["x"], g["W1"], g["A1"])
    r = ml.route_align(g["logits"], g["adapter_ids"], w.topk, d)
    want = ml.forward(g["x"], g["logits"], *_weights(g), g["adapter_ids"], w.topk)
    ws = ml.new_workspace(d, w.topk, DEV)
    ws.fill_(255)
    got = ml.forward_topk(g["x"], r["topk_ids"], r["topk_w"], *_weights(g), g["adapter_ids"], workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert ml.debug_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "tiled64"])
def test_e4m3_equals_the_layer_on_its_own_routing(name):
    w = SHAPES[name]
    g = _gpu(configs.make_inputs(w, 2))
    q = {}
    for n in ("W1", "W2"):
        f = g[n].float()
        s = f.abs().amax(-1).clamp_min(1e-20) / 448
        q[n] = (f / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
        q[n + "_scale"] = s.contiguous()
    d = ml.dims_of(g["x"], g["W1"], g["A1"])
    r = ml.route_align(g["logits"], g["adapter_ids"], w.topk, d)
    lora = [g[k] for k in ("A1", "B1", "A2", "B2")]
    want = ml.forward_fp8(g["x"], g["logits"], q["W1"], q["W1_scale"], q["W2"], q["W2_scale"], *lora,
                          g["adapter_ids"], w.topk)
    got = ml.forward_topk(g["x"], r["topk_ids"], r["topk_w"], q["W1"], q["W2"], *lora, g["adapter_ids"],
                          W1_scale=q["W1_scale"], W2_scale=q["W2_scale"])
    assert torch.equal(got, want)


def _choices(w, seed, empty):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, w.n_experts, (w.T, w.topk)).astype(np.int32)  # repeated experts among them
    ids[rng.random((w.T, w.topk)) < empty] = -1
    wt = rng.random((w.T, w.topk)).astype(np.float32) - 0.25
    return ids, wt


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("empty", [0.0, 0.4, 0.97])
def test_empty_slots_and_repeated_experts_match_the_oracle(name, empty):
    w = SHAPES[name]
    print("forward_topk oracle", name, empty, flush=True)
    inp = configs.make_inputs(w, 3)
    ids, wt = _choices(w, 5, empty)
    ids[0] = 0 if empty < 0.9 else -1
    g = _gpu(inp)
    wg = torch.from_numpy(wt.copy())
    wg[torch.from_numpy(ids) < 0] = float("nan")  # the weight of an empty slot is not used
    d = ml.dims_of(g["x"], g["W1"], g["A1"])
    ws = ml.new_workspace(d, w.topk, DEV)
    ws.fill_(255)
    y = ml.forward_topk(g["x"], torch.from_numpy(ids).to(DEV), wg.to(DEV), *_weights(g), g["adapter_ids"],
                        workspace=ws)
    torch.cuda.synchronize()
    ref = _reference(inp, ids, wt)
    check_close(y, ref, what=name)
    tab = ml.read_layout_tables(ws, d, w.topk)
    assert ml.debug_status(ws) == 0
    flat = ids.reshape(-1)
    np.testing.assert_array_equal(tab["pair_row"] < 0, flat < 0)
    live = np.nonzero(flat >= 0)[0]
    ad = inp["adapter_ids"].numpy()
    order = sorted(live.tolist(), key=lambda p: (flat[p], ad[p // w.topk], p))
    sp = tab["sorted_pairs"]
    np.testing.assert_array_equal(sp[sp >= 0], np.array(order, np.int32))
    np.testing.assert_array_equal(sp[tab["pair_row"][live]], live.astype(np.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHAPES)
def test_no_expert_at_all(name):
    w = SHAPES[name]
    print("forward_topk empty", name, flush=True)
    g = _gpu(configs.make_inputs(w, 4))
    ids = torch.full((w.T, w.topk), -1, dtype=torch.int32, device=DEV)
    y = torch.full((w.T, w.hidden), 7.0, dtype=BF, device=DEV)
    ml.forward_topk(g["x"], ids, torch.ones(w.T, w.topk, device=DEV), *_weights(g), g["adapter_ids"], y=y)
    torch.cuda.synchronize()
    assert (y == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "tiled64"])
def test_ids_out_of_range_are_empty_and_flagged(name):
    w = SHAPES[name]
    inp = configs.make_inputs(w, 6)
    g = _gpu(inp)
    ids, wt = _choices(w, 7, 0.1)
    bad = ids.copy()
    bad[3, 0], bad[5, 1], bad[7, 0] = w.n_experts, -2, 2 ** 30
    ids[3, 0] = ids[5, 1] = ids[7, 0] = -1
    d = ml.dims_of(g["x"], g["W1"], g["A1"])
    ws = ml.new_workspace(d, w.topk, DEV)
    wg = torch.from_numpy(wt).to(DEV)
    got = ml.forward_topk(g["x"], torch.from_numpy(bad).to(DEV), wg, *_weights(g), g["adapter_ids"], workspace=ws)
    assert ml.debug_status(ws) == ml.FLAG_EXPERT_RANGE
    want = ml.forward_topk(g["x"], torch.from_numpy(ids).to(DEV), wg, *_weights(g), g["adapter_ids"], workspace=ws)
    assert ml.debug_status(ws) == 0
    assert torch.equal(got, want)


def _block(g, s, topk, n_groups, topk_groups, mask, buf=None):
    """Router logits, expert choice, routed experts with their adapters, and the shared expert onto
    their output."""
    b = buf or {}
    logits = ml.router_logits(g["x"], s["W_router"], out=b.get("logits"))
    ids, wt = ml.route(logits, topk, scoring="sigmoid", bias=s["bias"], n_groups=n_groups, topk_groups=topk_groups,
                       group_score="top2", scale=1.5, token_mask=mask, topk_ids=b.get("ids"), topk_w=b.get("w"))
    routed = ml.forward_topk(g["x"], ids, wt, *_weights(g), g["adapter_ids"], y=b.get("routed"),
                             workspace=b.get("ws"))
    act = ml.linear(g["x"], s["Ws1"], act="swiglu", y=b.get("act"), workspace=b.get("ws1"))
    return ids, wt, ml.linear(act, s["Ws2"], residual=routed, y=b.get("y"), workspace=b.get("ws2"))


def _block_inputs(T):
    w = Workload("block", T, 256, 384, 16, 4, 5, 16)
    inp = configs.make_inputs(w, 8)
    gen = torch.Generator().manual_seed(T)
    shared = dict(W_router=(0.3 * torch.randn(16, 256, generator=gen)).to(BF), bias=0.1 * torch.randn(16, generator=gen),
                  Ws1=(0.05 * torch.randn(2 * 512, 256, generator=gen)).to(BF),
                  Ws2=(0.05 * torch.randn(256, 512, generator=gen)).to(BF))
    mask = torch.rand(T, generator=gen) < 0.8
    mask[0] = T == 1
    return w, inp, shared, mask


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 700])
def test_router_layer_and_shared_expert_together(T):
    w, inp, shared, mask = _block_inputs(T)
    print("block", T, flush=True)
    inp["x"] = (20 * inp["x"].float()).to(BF)
    g, s = _gpu(inp), {k: v.to(DEV) for k, v in shared.items()}
    ids, wt, y = _block(g, s, 4, 4, 2, mask.to(DEV))
    torch.cuda.synchronize()
    ids, wt = ids.cpu().numpy(), wt.cpu().numpy()
    # (the choice itself is checked elsewhere: here its results have to reach the layer)
    m = mask.numpy()
    assert (ids[~m] == -1).all() and (wt[~m] == 0).all() and (ids[m] >= 0).all()
    np.testing.assert_allclose(wt[m].sum(1), 1.5, rtol=1e-5)
    x = inp["x"].double()
    v = x @ shared["Ws1"].double().T
    act = (v[:, :512] * torch.sigmoid(v[:, :512]) * v[:, 512:])
    ref = _reference(inp, ids, wt) + (act @ shared["Ws2"].double().T).numpy()
    check_close(y, ref, what="block")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [24, 300])
def test_the_run_captured_and_replayed(T):
    """The whole run in a graph, replayed on new inputs with eager runs in between (which use
    workspaces of their own)."""
    w, inp, shared, mask = _block_inputs(T)
    g, s, m = _gpu(inp), {k: v.to(DEV) for k, v in shared.items()}, mask.to(DEV)
    d = ml.dims_of(g["x"], g["W1"], g["A1"])
    buf = dict(logits=torch.empty(T, 16, device=DEV), ids=torch.empty(T, 4, dtype=torch.int32, device=DEV),
               w=torch.empty(T, 4, device=DEV), routed=torch.empty(T, 256, dtype=BF, device=DEV),
               act=torch.empty(T, 512, dtype=BF, device=DEV), y=torch.empty(T, 256, dtype=BF, device=DEV),
               ws=ml.new_workspace(d, 4, DEV), ws1=torch.empty(64 << 20, dtype=torch.uint8, device=DEV),
               ws2=torch.empty(64 << 20, dtype=torch.uint8, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _block(g, s, 4, 4, 2, m, buf)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _block(g, s, 4, 4, 2, m, buf)
    for i in range(4):
        g["x"].copy_((0.2 * torch.randn(T, 256, device=DEV)).to(BF))
        m.copy_(torch.rand(T, device=DEV) < 0.7)
        for k in ("ids", "w", "y"):
            buf[k].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        ids, wt, y = _block(g, s, 4, 4, 2, m)
        assert torch.equal(buf["ids"], ids) and torch.equal(buf["w"], wt) and torch.equal(buf["y"], y), i


# ----------------------------------------------------------------------------- refusals (CPU)

def test_forward_topk_host_validation_without_device():
    lib = ml.lib()
    d = ml.Dims(16, 256, 512, 8, 4, 8)
    base = [0x10000 * (i + 1) for i in range(14)]
    # x, ids, w, W1, s1, W2, s2, A1, B1, A2, B2, adapter_ids, y, workspace

    def call(p, dd=d, topk=2, scales=False, ws=None):
        q = list(p)
        if not scales:
            q[4] = q[6] = None
        n = ml.workspace_size(dd, topk) if ws is None else ws
        return lib.moe_lora_forward_topk(*q[:12], topk, ctypes.byref(dd), q[12], q[13], n, None)

    for i in range(14):
        if i in (4, 6):
            continue
        p = list(base)
        p[i] = None
        assert call(p) == ml.ENULL, i
        if i < 13:
            p[i] = base[i] + 8
            assert call(p) == ml.EALIGN, i
    for i in (4, 6):
        p = list(base)
        p[i] = None
        assert call(p, scales=True) == ml.ENULL, i
        p[i] = base[i] + 2
        assert call(p, scales=True) == ml.EALIGN, i
    p = list(base)
    p[13] += 16
    assert call(p) == ml.EWORKSPACE
    assert call(base, ws=ml.workspace_size(d, 2) - 1) == ml.EWORKSPACE
    assert call(base, ml.Dims(16, 250, 512, 8, 4, 8)) == ml.EINVAL_DIMS
    assert call(base, topk=9) == ml.EINVAL_DIMS
    assert call([None] * 14, ml.Dims(0, 256, 512, 8, 4, 8)) == ml.OK
