"""Dense projection (moe_lora_linear) against float64. The bound per element: half a bf16 step of
the result, and the fp32 sum's error (K additions of at most 2^-24 of the sum of magnitudes each)
through the activation, with 2^-18 of the value for the fp32 epilogue (exponential, division)."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import lora_mixture_experts_amd as ml

DEV = "cuda"
BF = torch.bfloat16


def _decode(W, scale):
    return W.double() if scale is None else W.view(torch.float8_e4m3fn).double() * scale.double()[:, None]


def _reference(x, W, scale, bias, act, residual):
    """(y, bound) in float64 on the inputs' device."""
    xd, Wd = x.double(), _decode(W, scale)
    v = xd @ Wd.T
    mag = xd.abs() @ Wd.abs().T
    if bias is not None:
        v = v + bias.double()
        mag = mag + bias.double().abs()
    dv = (x.shape[1] + 4) * 2.0 ** -24 * mag
    if act == "swiglu":
        N = W.shape[0] // 2
        g, u, dg, du = v[:, :N], v[:, N:], dv[:, :N], dv[:, N:]
        y = g * torch.sigmoid(g) * u
        dy = 1.1 * dg * (u.abs() + du) + g.abs() * du
    else:
        y = {"none": lambda: v, "relu": lambda: v.clamp_min(0), "silu": lambda: v * torch.sigmoid(v),
             "gelu": lambda: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
             "gelu_tanh": lambda: v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))}[act]()
        dy = 1.2 * dv  # no activation is steeper than 1.13
    dy = dy + 2.0 ** -18 * y.abs()
    if residual is not None:
        y = y + residual.double()
    return y, dy + 2.0 ** -8 * (y.abs() + dy) + 2.0 ** -126


def _inputs(T, K, N, act, w, seed, bias=True, residual=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    Wf = torch.randn(rows, K, generator=g, device=DEV) / math.sqrt(K)
    scale = None
    W = Wf.to(BF)
    if w == "e4m3":
        scale = (Wf.abs().amax(1) / 448).clamp_min(1e-20)
        W = (Wf / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    b = torch.randn(rows, generator=g, device=DEV).to(BF) if bias else None
    r = torch.randn(T, N, generator=g, device=DEV).to(BF) if residual else None
    return x, W, scale, b, r


def _compare(y, x, W, scale, b, act, r):
    ref, bound = _reference(x, W, scale, b, act, r)
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    worst = (err / bound).max().item()
    assert worst <= 1.0, worst


def _check(T, K, N, act, w, bias=True, residual=True, seed=0):
    print("linear", T, K, N, act, w, bias, residual, flush=True)
    x, W, scale, b, r = _inputs(T, K, N, act, w, seed + T + K + N, bias, residual)
    y = ml.linear(x, W, w_scale=scale, bias=b, act=act, residual=r)
    torch.cuda.synchronize()
    _compare(y, x, W, scale, b, act, r)
    assert torch.equal(y, ml.linear(x, W, w_scale=scale, bias=b, act=act, residual=r)), "not the same bits twice"
    return y


SHAPES = [
    # T, K, N: one token to prompts; nothing, some or all of it a multiple of a tile
    (1, 16, 1), (1, 128, 64), (1, 4096, 256), (2, 48, 17), (15, 1024, 130), (16, 64, 16), (17, 112, 33),
    (31, 2000, 65), (32, 512, 512), (33, 656, 100), (48, 1024, 257), (64, 2048, 96), (65, 128, 64), (65, 80, 3),
    (100, 1040, 131), (129, 2048, 384), (200, 16, 129), (256, 64, 1000), (300, 176, 2050), (513, 1024, 255),
    (777, 2032, 531), (1500, 320, 1030), (2100, 256, 4200),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3"), ("swiglu", "e4m3")])
def test_linear_matches_float64(T, K, N, act, w):
    _check(T, K, N, act, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 8, 5), (40, 24, 70), (90, 1000, 140), (600, 4088, 260)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_rows_of_8_elements(T, K, N, act):
    """bf16 rows need be a multiple of 8 only."""
    _check(T, K, N, act, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_linear_epilogues(T, act, bias, residual):
    _check(T, 256, 192, act, "bf16", bias, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(7, 512, 100), (130, 512, 100), (520, 528, 203)])
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3")])
def test_linear_strided_rows(T, K, N, act, w):
    """x, W, residual and y inside wider buffers, whose other columns hold NaN and stay untouched;
    residual and y at odd strides and offsets."""
    x, W, scale, b, r = _inputs(T, K, N, act, w, 11)

    def inside(t, left, right):
        wide = torch.full((t.shape[0] + 1, left + t.shape[1] + right), float("nan") if t.dtype == BF else 127,
                          dtype=t.dtype, device=DEV)
        view = wide[:-1, left:left + t.shape[1]]
        view.copy_(t)
        return wide, view

    xw, xv = inside(x, 8, 24)
    Ww, Wv = inside(W, 16, 32)
    for left, right in ((3, 2), (4, 4)):
        rw, rv = inside(r, left, right)
        yw, yv = inside(torch.zeros(T, N, dtype=BF, device=DEV), left + 1, right)
        keep = yw.clone()
        out = ml.linear(xv, Wv, w_scale=scale, bias=b, act=act, residual=rv, y=yv)
        torch.cuda.synchronize()
        _compare(out, x, W, scale, b, act, r)
        keep[:-1, left + 1:left + 1 + N] = out
        assert torch.equal(torch.nan_to_num(keep, 9.0), torch.nan_to_num(yw, 9.0))


@pytest.mark.gpu
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3")])
def test_linear_one_row_of_any_stride(act, w):
    """The stride of a single row is never stepped: one token of a long sequence for x, the residual
    and y, rows of buffers whose width is no multiple of 16 bytes, a W of one row."""
    K, N = 512, 96
    x, W, scale, b, r = _inputs(1, K, N, act, w, 61)

    def last(t):  # the last position of a sequence [1][S][n]
        n = t.shape[1]
        seq = torch.zeros(1, (1 << 22) // n + 2, n, dtype=t.dtype, device=DEV)
        seq[:, -1] = t
        assert seq[:, -1].stride(0) >= 1 << 22
        return seq[:, -1]

    def odd(t):  # the first row of a buffer of odd width
        wide = torch.zeros(3, t.shape[1] + 3, dtype=t.dtype, device=DEV)
        wide[:1, :t.shape[1]] = t
        return wide[:1, :t.shape[1]]

    for place in (last, odd):
        y = place(torch.zeros(1, N, dtype=BF, device=DEV))
        assert ml.linear(place(x), W, w_scale=scale, bias=b, act=act, residual=place(r), y=y) is y
        _compare(y, x, W, scale, b, act, r)
    if act == "none":
        one = ml.linear(place(x), place(W[:1]), w_scale=None if scale is None else scale[:1], bias=b[:1])
        _compare(one, x, W[:1], None if scale is None else scale[:1], b[:1], act, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(5, 96), (150, 96), (1100, 1000)])
def test_linear_onto_its_residual(T, N):
    x, W, _, b, r = _inputs(T, 512, N, "gelu", "bf16", 21)
    want = ml.linear(x, W, bias=b, act="gelu", residual=r)
    y = r.clone()
    assert ml.linear(x, W, bias=b, act="gelu", residual=y, y=y) is y
    assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 100, 600])
def test_linear_poisoned_workspace_and_other_streams(T):
    """The workspace needs no initialisation; a call on another stream gives the same bits."""
    K, N = 2048, 256
    x, W, _, b, r = _inputs(T, K, N, "swiglu", "bf16", 31)
    want = ml.linear(x, W, bias=b, act="swiglu", residual=r)
    d = ml.LinearDims(T, K, N, ml.ACTIVATIONS["swiglu"], 0, K, K, N, N)
    need = ml.lib().moe_lora_linear_workspace_size(ctypes.byref(d))
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = ml.linear(x, W, bias=b, act="swiglu", residual=r, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert (ws[need:] == 255).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 100])
def test_linear_infinities_stay_in_their_rows(T):
    x, W, _, _, _ = _inputs(T, 256, 80, "none", "bf16", 41)
    want = ml.linear(x, W)
    x2 = x.clone()
    x2[1, 5] = math.inf
    x2[2, 7] = math.nan
    y = ml.linear(x2, W)
    rows = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[rows], want[rows])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "swiglu"])
def test_linear_large_arguments(T, act):
    """Activations run into their limits, never into NaN."""
    x = torch.full((T, 64), 100.0, dtype=BF, device=DEV)
    x[1] = -100.0
    W = torch.ones(32, 64, dtype=BF, device=DEV)
    y = ml.linear(x, W, act=act).double()
    assert torch.isfinite(y).all()
    if act == "swiglu":
        assert (y[0] == float(torch.tensor(6400.0 ** 2).to(BF))).all() and (y[1] == 0).all()
    else:
        assert (y[0] == 6400.0).all() and (y[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 200])
def test_linear_graph_replays(T):
    """Captured with a workspace of its own; eager calls between the replays change nothing."""
    K, N = 2048, 192
    x, W, _, b, r = _inputs(T, K, N, "swiglu", "bf16", 51)
    y = torch.empty(T, N, dtype=BF, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ml.linear(x, W, bias=b, act="swiglu", residual=r, y=y, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ml.linear(x, W, bias=b, act="swiglu", residual=r, y=y, workspace=ws)
    for i in range(4):
        x.copy_(torch.randn(T, K, device=DEV).to(BF))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ml.linear(x, W, bias=b, act="swiglu", residual=r)), i


@pytest.mark.gpu
@pytest.mark.parametrize("T", [12, 40, 96])
def test_linear_weights_past_4_gib(T):
    """Weight rows whose byte offsets pass 32 bits: the last rows of a 5 GiB matrix (4 GiB between
    gate and up)."""
    K, rows = 4096, 600000
    W = torch.zeros(rows, K, dtype=BF, device=DEV)
    tail = torch.randn(300, K, device=DEV).to(BF)
    W[-300:] = tail
    W[rows // 2 - 300:rows // 2] = tail
    x = torch.randn(T, K, device=DEV).to(BF)
    y = ml.linear(x, W)
    _compare(y[:, -300:], x, tail, None, None, "none", None)
    assert (y[:, :rows // 2 - 300] == 0).all()
    y2 = ml.linear(x, W, act="swiglu")
    _compare(y2[:, -300:], x, torch.cat([tail, tail]), None, None, "swiglu", None)


@pytest.mark.gpu
def test_linear_and_route_from_two_threads():
    """Two threads, each on a stream of its own, split and whole forms: the same bits as alone."""
    x, W, _, b, r = _inputs(100, 2064, 131, "silu", "bf16", 91)
    assert ml.linear_plan(100, 2064, 131, "silu")["splits"] > 1
    x2, W2, s2, b2, _ = _inputs(300, 1040, 515, "none", "e4m3", 92, True, False)
    logits, bias = torch.randn(700, 96, device=DEV), 0.1 * torch.randn(96, device=DEV)

    def calls():
        ids, w = ml.route(logits, 6, scoring="sigmoid", bias=bias, n_groups=8, topk_groups=3, group_score="top2")
        return ml.linear(x, W, bias=b, act="silu", residual=r), ml.linear(x2, W2, w_scale=s2, bias=b2), ids, w

    want = calls()
    torch.cuda.synchronize()
    right = []

    def work():
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(200):
                got = calls()
                side.synchronize()
                right.append(all(torch.equal(g, v) for g, v in zip(got, want)))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(right) == 400 and all(right)


@pytest.mark.gpu
def test_linear_empty_batch():
    W = torch.zeros(24, 16, dtype=BF, device=DEV)
    assert ml.linear(torch.empty(0, 16, dtype=BF, device=DEV), W).shape == (0, 24)


# Sizes that take each tile of the tiled kernel, with and without splits of the reduction: (T, K, N, tile
# rows, tile columns, split), the same for bf16 and E4M3. Rows, columns and K are no multiple of a tile or
# of a step; the last of each list reads more than 128 MB of bf16 weights in one row tile.
FORMS = [(131, 784, 203, 64, 64, False), (67, 4112, 257, 64, 64, True), (257, 528, 4203, 64, 128, False),
         (40, 4112, 4203, 64, 128, True), (1500, 528, 1301, 128, 128, False), (2051, 3088, 131, 128, 128, True),
         (3000, 528, 4203, 256, 256, False), (3000, 4112, 1301, 256, 256, True), (40, 4112, 17003, 64, 128, False)]
SWIGLU_FORMS = [(131, 784, 203, 64, 64, False), (67, 4112, 257, 64, 64, True), (403, 1040, 2101, 64, 128, False),
                (40, 4112, 4203, 64, 128, True), (257, 528, 4203, 128, 128, False), (67, 3088, 2050, 128, 128, True),
                (3000, 528, 2101, 256, 256, False), (193, 8208, 4203, 256, 256, True), (40, 4112, 8501, 64, 128, False)]


def _assert_form(T, K, N, rows, cols, split, act, w):
    p = ml.linear_plan(T, K, N, act, w == "e4m3")
    groups = {(64, 64): 4, (64, 128): 2}.get((rows, cols), 1)
    assert (p["streamed"], p["tile_rows"], p["tile_cols"], p["k_groups"]) == (0, rows, cols, groups)
    assert (p["splits"] > 1) == split


@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_linear_plan_of_every_form(w):
    """The sizes that the tests of the tiled kernel's forms are made for still take them."""
    for form in FORMS:
        for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
            _assert_form(*form, act, w)
    for form in SWIGLU_FORMS:
        _assert_form(*form, "swiglu", w)
    one = ml.linear_plan(1, 4096, 4096, e4m3=w == "e4m3")
    assert one == dict(streamed=1, tile_rows=0, tile_cols=0, k_groups=0, splits=1)


def test_linear_plan_refuses():
    for bad in (dict(T=-1), dict(in_features=508), dict(out_features=1 << 22), dict(T=(1 << 30) - 1, out_features=1 << 20)):
        f = dict(T=100, in_features=512, out_features=64)
        f.update(bad)
        with pytest.raises(ml.MoeLoraError) as e:
            ml.linear_plan(**f)
        assert e.value.code == ml.EINVAL_DIMS
    with pytest.raises(ValueError):
        ml.linear_plan(1, 16, 16, "tanh")
    d = ml.LinearDims(100, 512, 64, 0, 0, 512, 512, 64, 64)
    assert ml.lib().moe_lora_linear_plan(ctypes.byref(d), None) == ml.ENULL
    assert ml.lib().moe_lora_linear_plan(None, ctypes.byref(ml.LinearPlanInfo())) == ml.ENULL


def _acts(forms, acts, split):
    return [(*f, a) for f in forms for a in acts if f[-1] == split]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,K,N,rows,cols,split,act", _acts(FORMS, ACTS, True) + _acts(SWIGLU_FORMS, ("swiglu",), True))
def test_linear_split_forms(T, K, N, rows, cols, split, act, w):
    """Splits of every tile (a wavefront of the 256 x 256 one writes its sums 32 rows at a time through
    the same LDS), and every activation in the launch that adds them."""
    _assert_form(T, K, N, rows, cols, split, act, w)
    _check(T, K, N, act, w)


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,K,N,rows,cols,split,act", _acts(FORMS, ACTS, False) + _acts(SWIGLU_FORMS, ("swiglu",), False))
def test_linear_whole_forms(T, K, N, rows, cols, split, act, w):
    """Every tile without splits: several turns of the LDS ring, a partial last step, each activation."""
    _assert_form(T, K, N, rows, cols, split, act, w)
    _check(T, K, N, act, w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,rows,cols,split,act", _acts(FORMS, ("silu",), False) + _acts(FORMS, ("none",), True)
                         + _acts(SWIGLU_FORMS, ("swiglu",), False) + _acts(SWIGLU_FORMS, ("swiglu",), True))
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_linear_forms_without_operands(T, K, N, rows, cols, split, act, bias, residual):
    _assert_form(T, K, N, rows, cols, split, act, "bf16")
    _check(T, K, N, act, "bf16", bias, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,rows,cols,split,act", _acts(FORMS, ("gelu",), False) + _acts(FORMS, ("gelu",), True)
                         + _acts(SWIGLU_FORMS, ("swiglu",), False) + _acts(SWIGLU_FORMS, ("swiglu",), True))
def test_linear_forms_onto_the_residual(T, K, N, rows, cols, split, act):
    """y in place of the residual, inside a wider buffer whose other columns stay."""
    _assert_form(T, K, N, rows, cols, split, act, "bf16")
    x, W, _, b, r = _inputs(T, K, N, act, "bf16", 81)
    wide = torch.full((T, N + 5), 7.0, dtype=BF, device=DEV)
    y = wide[:, 3:3 + N]
    y.copy_(r)
    assert ml.linear(x, W, bias=b, act=act, residual=y, y=y) is y
    _compare(y, x, W, None, b, act, r)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + N:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 131, 3000])
def test_linear_decodes_every_e4m3_code(T):
    """All 256 codes, one a weight row, against torch's decoding: NaN codes give NaN, in their column only."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    W = torch.zeros(256, 528, dtype=torch.uint8, device=DEV)
    W[:, 517] = codes
    x = torch.zeros(T, 528, dtype=BF, device=DEV)
    x[:, 517] = 1.0
    y = ml.linear(x, W, w_scale=torch.ones(256, device=DEV)).float()
    want = codes.view(torch.float8_e4m3fn).float().expand(T, 256)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.isnan(want).sum() == 2 * T
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))


# ----------------------------------------------------------------------------- refusals (CPU)

FIELDS = dict(T=100, in_features=512, out_features=64, act=0, w_type=0, x_stride=512, w_stride=512, y_stride=64,
              residual_stride=64)
PTRS = dict(x=0x100000, W=0x200000, w_scale=None, bias=0x300000, residual=0x400000, y=0x500000, ws=0x600000)


def _call(ws_bytes=1 << 40, ptrs=None, **kw):
    p = dict(PTRS)
    p.update(ptrs or {})
    d = ml.LinearDims(**{**FIELDS, **kw})
    return ml.lib().moe_lora_linear(p["x"], p["W"], p["w_scale"], p["bias"], p["residual"], ctypes.byref(d),
                                    p["y"], p["ws"], ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 30), dict(in_features=0), dict(in_features=508), dict(out_features=0), dict(act=6), dict(act=-1),
    dict(w_type=2), dict(x_stride=504), dict(x_stride=516), dict(w_stride=500), dict(w_stride=516),
    dict(y_stride=63), dict(residual_stride=63), dict(x_stride=1 << 22), dict(w_stride=1 << 22),
    dict(y_stride=1 << 22), dict(w_type=1, in_features=504, w_stride=512), dict(w_type=1, w_stride=520)])
def test_linear_refuses_fields_out_of_range(bad):
    scale = {"w_scale": 0x700000} if bad.get("w_type") == 1 else {}
    assert _call(ptrs=scale, **bad) == ml.EINVAL_DIMS
    if "residual_stride" not in bad:
        d = ml.LinearDims(**{**FIELDS, **bad})
        assert ml.lib().moe_lora_linear_workspace_size(ctypes.byref(d)) == 0


def test_linear_refuses_pointers():
    for name in ("x", "W", "y"):
        assert _call(ptrs={name: None}) == ml.ENULL
    assert _call(ptrs={"w_scale": None}, w_type=1) == ml.ENULL
    assert _call(ptrs={"w_scale": 0x700000}) == ml.EUNSUPPORTED
    for name, off in (("x", 8), ("W", 8), ("bias", 1), ("residual", 1), ("y", 1)):
        assert _call(ptrs={name: PTRS[name] + off}) == ml.EALIGN, name
    assert _call(ptrs={"w_scale": 0x700002}, w_type=1) == ml.EALIGN
    assert ml.lib().moe_lora_linear(*[0x100000] * 5, None, 0x100000, None, 0, None) == ml.ENULL
    assert _call(T=0, ptrs={k: None for k in PTRS}) == ml.OK


def test_linear_refuses_more_tiles_than_a_launch_holds():
    big = dict(T=(1 << 30) - 1, out_features=1 << 20, y_stride=1 << 20, residual_stride=1 << 20)
    assert _call(**big) == ml.EINVAL_DIMS


def test_linear_refuses_workspaces():
    big = dict(T=100, in_features=8192, x_stride=8192, w_stride=8192)
    d = ml.LinearDims(**{**FIELDS, **big})
    need = ml.lib().moe_lora_linear_workspace_size(ctypes.byref(d))
    assert need > 0 and need % 256 == 0
    assert _call(ws_bytes=need - 1, **big) == ml.EWORKSPACE
    assert _call(ptrs={"ws": PTRS["ws"] + 16}, **big) == ml.EWORKSPACE
    assert _call(ptrs={"ws": None}, **big) == ml.ENULL


def test_linear_binding_refuses():
    x, W = torch.zeros(4, 16, dtype=BF), torch.zeros(8, 16, dtype=BF)
    with pytest.raises(ValueError):
        ml.linear(x, W)
    with pytest.raises(ValueError):
        ml.linear(x, W, act="tanh")
    with pytest.raises(ValueError):
        ml.linear(x[0], W)


@pytest.mark.gpu
def test_linear_refuses_outputs_over_inputs():
    """An output that shares bytes with x, W or a residual it is not in place of is refused; column
    slices of one buffer share none."""
    buf = torch.randn(8, 256, device=DEV).to(BF)
    W = torch.randn(64, 64, device=DEV).to(BF)
    x, y = buf[:, :64], buf[:, 64:128]
    want = ml.linear(x, W)
    flat = torch.empty(64 * 64 * 2, dtype=BF, device=DEV)
    over = [(x, W, None, x), (x, W, flat[:512].view(8, 64), flat[64:576].view(8, 64)),
            (x, W, buf[:, 64:128], buf.view(-1)[64:576].view(8, 64)), (x, flat[:4096].view(64, 64), None, flat[4032:4544].view(8, 64))]
    for a, w, residual, out in over:
        with pytest.raises(ValueError):
            ml.linear(a, w, residual=residual, y=out)
    assert torch.equal(ml.linear(x, W, y=y), want)
    one = buf[:1, :64].clone()
    assert torch.equal(ml.linear(x[:1], W, residual=one, y=one), one)


@pytest.mark.gpu
def test_linear_refuses_every_shared_byte():
    """y in column slices that meet an input's, over a bias, a scale or a workspace in use; slices that
    share no byte are taken, whatever their strides."""
    buf = torch.randn(16, 256, device=DEV).to(BF)
    W = torch.randn(64, 64, device=DEV).to(BF)
    x = buf[:8, :64]
    want = ml.linear(x, W)
    for y in (buf[:8, 32:96], buf[1:9, :64], buf[:8, 63:127], buf[::2, 8:72], buf.view(-1)[:8 * 320].view(8, 320)[:, 64:128]):
        with pytest.raises(ValueError, match="overlaps"):
            ml.linear(x, W, y=y)
    for y in (buf[:8, 64:128], buf[8:, :64], buf[::2, 64:128], buf[1::2, 192:]):
        assert torch.equal(ml.linear(x, W, y=y), want)
    r = torch.randn(8, 64, device=DEV).to(BF)
    with pytest.raises(ValueError, match="overlaps"):
        ml.linear(r, W, residual=buf[:8, :64], y=buf[:8, 8:72])
    line = torch.zeros(8 * 64 + 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        ml.linear(r, W, bias=line[448:512], y=line[:512].view(8, 64))
    codes = torch.zeros(64, 64, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        ml.linear(r, codes, w_scale=line.view(torch.float32)[224:288], y=line[:512].view(8, 64))
    assert torch.equal(ml.linear(r, W, bias=line[512:], y=line[:512].view(8, 64)), ml.linear(r, W))

    # a workspace counts where the call uses one, and as far as it does
    T, K, N = 100, 8192, 64
    x, W, _, b, _ = _inputs(T, K, N, "none", "bf16", 71, True, False)
    d = ml.LinearDims(T, K, N, 0, 0, K, K, N, N)
    need = ml.lib().moe_lora_linear_workspace_size(ctypes.byref(d))
    assert need > 0
    ws = torch.empty(need + T * N * 2, dtype=torch.uint8, device=DEV)
    behind = ws[need:].view(BF).view(T, N)
    assert torch.equal(ml.linear(x, W, bias=b, y=behind, workspace=ws), ml.linear(x, W, bias=b))
    within = ws[need - 16:need - 16 + T * N * 2].view(BF).view(T, N)
    with pytest.raises(ValueError, match="overlaps"):
        ml.linear(x, W, bias=b, y=within, workspace=ws)
    with pytest.raises(ValueError, match="overlaps"):
        ml.linear(x, W, bias=b, workspace=x.view(-1).view(torch.uint8))
    few, part = x[:1, :512], W[:, :512]
    d = ml.LinearDims(1, 512, N, 0, 0, 512, K, N, N)
    assert ml.lib().moe_lora_linear_workspace_size(ctypes.byref(d)) == 0
    assert torch.equal(ml.linear(few, part, bias=b, workspace=x.view(-1).view(torch.uint8)), ml.linear(few, part, bias=b))
