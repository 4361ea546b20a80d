"""Dense projection with a batch's adapters in its epilogue (moe_lora_linear_lora) against float64. The
bound per element: half a bf16 step of the result, and through the activation the fp32 errors of the base
sum (K additions of at most 2^-24 of the sum of magnitudes each), of z (K additions, carried on by |B|), of
z as two bf16 (2^-8 of 2^-8 of it) and of the 2 r additions behind it."""
import ctypes
import math
import threading

import pytest
import torch

import lora_mixture_experts_amd as ml
from tests.test_linear import BF, DEV, FORMS, SWIGLU_FORMS, _inputs

NONE = ("none", "bf16")


def _decode(W, scale):
    return W.double() if scale is None else W.view(torch.float8_e4m3fn).double() * scale.double()[:, None]


def _adapters(nA, r, K, rows, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 7)
    A = (torch.randn(nA, r, K, generator=g, device=DEV) / math.sqrt(K)).to(BF)
    return A, torch.randn(nA, rows, r, generator=g, device=DEV).to(BF)


def _ids(T, nA, pattern, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    if pattern == "random":  # -1 among them
        ids = torch.randint(-1, nA, (T,), generator=g)
    elif pattern == "runs":
        ids = (torch.arange(T) // 37 * 5 + 1) % (nA + 1) - 1
    elif pattern == "distinct":
        ids = torch.arange(T) % nA
    elif pattern == "one":
        ids = torch.full((T,), nA - 1)
    else:
        ids = torch.full((T,), -1)
    return ids.int().to(DEV)


def _reference(x, W, scale, b, act, res, A, B, ids):
    """(y, bound) in float64."""
    xd, Wd = x.double(), _decode(W, scale)
    K, r = x.shape[1], A.shape[1]
    v, mag = xd @ Wd.T, xd.abs() @ Wd.abs().T
    dv = (K + 4) * 2.0 ** -24 * mag
    idl = ids.tolist()
    for a in sorted({i for i in idl if 0 <= i < A.shape[0]}):
        rows = torch.tensor([t for t, i in enumerate(idl) if i == a], device=DEV)
        Ad, Bd = A[a].double(), B[a].double()
        z = xd[rows] @ Ad.T
        dz = (K + 4) * 2.0 ** -24 * (xd[rows].abs() @ Ad.abs().T) + 2.0 ** -16 * z.abs()
        v[rows] += z @ Bd.T
        dv[rows] += dz @ Bd.abs().T + (2 * r + 2) * 2.0 ** -24 * (z.abs() @ Bd.abs().T)
    if b is not None:
        v = v + b.double()
    dv = dv + 2.0 ** -22 * v.abs()
    if act == "swiglu":
        N = W.shape[0] // 2
        g, u, dg, du = v[:, :N], v[:, N:], dv[:, :N], dv[:, N:]
        y = g * torch.sigmoid(g) * u
        dy = 1.1 * dg * (u.abs() + du) + g.abs() * du
    else:
        y = {"none": lambda: v, "relu": lambda: v.clamp_min(0), "silu": lambda: v * torch.sigmoid(v),
             "gelu": lambda: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
             "gelu_tanh": lambda: v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))}[act]()
        dy = 1.2 * dv
    dy = dy + 2.0 ** -18 * y.abs()
    if res is not None:
        y = y + res.double()
    return y, dy + 2.0 ** -8 * (y.abs() + dy) + 2.0 ** -126


def _compare(y, *case):
    ref, bound = _reference(*case)
    assert torch.isfinite(y).all()
    worst = ((y.double() - ref).abs() / bound).max().item()
    assert worst <= 1.0, worst


def _check(T, K, N, act, w, r, nA, pattern, bias=True, residual=True, seed=0):
    print("linear_lora", T, K, N, act, w, r, nA, pattern, bias, residual, flush=True)
    x, W, scale, b, res = _inputs(T, K, N, act, w, seed + T + K + N, bias, residual)
    A, B = _adapters(nA, r, K, W.shape[0], seed)
    ids = _ids(T, nA, pattern, seed)
    y = ml.linear_lora(x, W, A, B, ids, w_scale=scale, bias=b, act=act, residual=res)
    torch.cuda.synchronize()
    _compare(y, x, W, scale, b, act, res, A, B, ids)
    again = ml.linear_lora(x, W, A, B, ids, w_scale=scale, bias=b, act=act, residual=res)
    assert torch.equal(y, again), "not the same bits twice"


SHAPES = [
    # T, K, N, rank, adapters, pattern: one token to prompts, odd rows and columns
    (1, 16, 1, 8, 1, "one"), (1, 4096, 256, 16, 4, "one"), (2, 48, 17, 64, 3, "random"), (15, 1024, 130, 8, 3, "random"),
    (16, 64, 16, 32, 20, "distinct"), (17, 112, 33, 16, 5, "random"), (31, 2000, 65, 64, 40, "distinct"),
    (32, 512, 512, 8, 2, "runs"), (33, 656, 100, 32, 9, "random"), (48, 1024, 257, 16, 48, "distinct"),
    (64, 2048, 96, 16, 7, "random"), (64, 2048, 96, 64, 64, "distinct"), (65, 128, 64, 16, 70, "distinct"),
    (100, 1040, 131, 8, 6, "random"), (129, 2048, 384, 64, 3, "runs"), (200, 16, 129, 32, 200, "distinct"),
    (256, 64, 1000, 16, 64, "random"), (513, 1024, 255, 8, 12, "runs"), (777, 2032, 531, 32, 5, "random"),
    (1500, 320, 1030, 16, 33, "runs"), (2100, 256, 4200, 64, 6, "runs"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,nA,pattern", SHAPES)
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3"), ("swiglu", "e4m3")])
def test_linear_lora_matches_float64(T, K, N, r, nA, pattern, act, w):
    _check(T, K, N, act, w, r, nA, pattern)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,nA,pattern", [
    (511, 528, 96, 16, 600, "random"), (512, 1024, 200, 32, 1024, "distinct"), (160, 1040, 64, 8, 5, "random"),  # by adapter
    (161, 1040, 64, 64, 5, "one"), (40, 512, 64, 16, 4, "random"), (512, 1040, 64, 8, 1, "one"), (511, 4096, 64, 64, 1000, "one"),
    (513, 528, 96, 16, 600, "random"), (300, 640, 96, 64, 1025, "random"), (33, 2048, 64, 16, 5000, "distinct"),  # by token
    (2100, 272, 300, 64, 50, "random"), (3000, 2064, 70, 32, 31, "runs"), (3, 16384, 33, 64, 2, "random"),
])
def test_linear_lora_shrink_forms(T, K, N, r, nA, pattern):
    """Both forms of the shrink on both sides of their borders, with K split and whole."""
    _check(T, K, N, "none", "bf16", r, nA, pattern)


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(16, 1), (80, 17), (1008, 250), (1024, 1000), (4096, 48), (8192, 33), (8208, 16), (1024, 4112)])
@pytest.mark.parametrize("r", [8, 16, 32, 64])
@pytest.mark.parametrize("act,w", [("gelu", "bf16"), ("swiglu", "bf16"), ("none", "e4m3"), ("swiglu", "e4m3")])
def test_linear_lora_one_token(K, N, r, act, w):
    """In one launch and in two, with an adapter, without one, and beside an adapter of NaNs."""
    for pattern in ("one", "none"):
        _check(1, K, N, act, w, r, 3, pattern)
    x, W, scale, _, _ = _inputs(1, K, N, act, w, 5, False, False)
    A, B = _adapters(3, r, K, W.shape[0], 5)
    ids = _ids(1, 2, "one")
    y = ml.linear_lora(x, W, A, B, ids, w_scale=scale, act=act)
    A[2], B[0] = math.nan, math.inf
    assert torch.equal(y, ml.linear_lora(x, W, A, B, ids, w_scale=scale, act=act))


@pytest.mark.gpu
def test_linear_lora_rows_far_apart():
    """Rows of x that lie 2^22 - 8 elements apart: offsets past 32 bits within a batch."""
    T, K, N = 300, 256, 64
    x, W, _, _, _ = _inputs(T, K, N, "none", "bf16", 91)
    A, B = _adapters(20, 16, K, N, 91)
    ids = _ids(T, 20, "random")
    wide = torch.empty(T, (1 << 22) - 8, dtype=BF, device=DEV)
    wide[:, 8:8 + K] = x
    y = ml.linear_lora(wide[:, 8:8 + K], W, A, B, ids)
    _compare(y, x, W, None, None, "none", None, A, B, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("act,w", [("gelu", "bf16"), ("swiglu", "bf16"), ("silu", "e4m3"), ("swiglu", "e4m3")])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_linear_lora_every_form(form, act, w):
    """Every tile of the tiled kernel, with and without splits of the reduction."""
    T, K, N, rows, cols, split = (SWIGLU_FORMS if act == "swiglu" else FORMS)[form]
    p = ml.linear_lora_plan(T, K, N, 9, 16, act, w == "e4m3")
    assert (p["streamed"], p["tile_rows"], p["tile_cols"], p["splits"] > 1) == (0, rows, cols, split)
    _check(T, K, N, act, w, 16, 9, "random")
    _check(T, K, N, act, w, 64, 4, "runs", bias=False, residual=False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 150])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_linear_lora_epilogues(T, act, bias, residual):
    _check(T, 256, 192, act, "bf16", 16, 5, "random", bias, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 8, 5), (40, 24, 70), (90, 1000, 140), (600, 4088, 260)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_lora_rows_of_8_elements(T, K, N, act):
    _check(T, K, N, act, "bf16", 8, 3, "random")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 512, 96), (20, 512, 96), (60, 1024, 320), (150, 512, 96), (1100, 256, 1000)])
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("gelu", "e4m3")])
def test_linear_lora_without_adapters_equals_linear(T, K, N, act, w):
    """No token with an adapter: the projection's bits, up to the place of the scale in split sums."""
    x, W, scale, b, r = _inputs(T, K, N, act, w, 5)
    A, B = _adapters(2, 16, K, W.shape[0], 5)
    A.fill_(math.nan)
    B.fill_(math.inf)
    ids = _ids(T, 2, "none")
    y = ml.linear_lora(x, W, A, B, ids, w_scale=scale, bias=b, act=act, residual=r)
    _compare(y, x, W, scale, b, act, r, A, B, ids)
    if w == "bf16":
        assert torch.equal(y, ml.linear(x, W, w_scale=scale, bias=b, act=act, residual=r))


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(2, 64), (30, 64), (64, 100), (150, 200), (2000, 1000)])
@pytest.mark.parametrize("pattern", ["random", "runs", "distinct"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_linear_lora_broken_adapter_stays_with_its_tokens(T, N, pattern, bad):
    """Infinities and NaNs in one adapter's A, another's B and in a token's row reach no other token."""
    K, nA, r = 256, 6, 16
    x, W, _, _, _ = _inputs(T, K, N, "none", "bf16", 71)
    A, B = _adapters(nA, r, K, N, 71)
    ids = _ids(T, nA, pattern, 3)
    want = ml.linear_lora(x, W, A, B, ids)
    A2, B2, x2 = A.clone(), B.clone(), x.clone()
    A2[1, 3, 7] = bad
    B2[2, 5, 1] = bad
    x2[0, 9] = bad
    y = ml.linear_lora(x2, W, A2, B2, ids)
    keep = (ids != 1) & (ids != 2)
    keep[0] = False
    assert torch.equal(y[keep], want[keep])
    assert not torch.isfinite(y[0]).any()
    two = ids == 2
    two[0] = False
    assert not torch.isfinite(y[two][:, 5]).any()
    cols = [c for c in range(N) if c != 5]
    assert torch.equal(y[two][:, cols], want[two][:, cols])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_linear_lora_adapter_ids_out_of_range(T):
    """Taken as none, and told by the workspace's flags."""
    K, N, nA = 512, 96, 3
    x, W, _, _, _ = _inputs(T, K, N, "none", "bf16", 81)
    A, B = _adapters(nA, 8, K, N, 81)
    ids = _ids(T, nA, "random", 2)
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)
    want = ml.linear_lora(x, W, A, B, ids, workspace=ws)
    assert ml.debug_status(ws) == 0
    bad = torch.where(ids == -1, nA + 5, ids)
    bad[T - 1] = -2
    fine = ids.clone()
    fine[T - 1] = -1
    want = ml.linear_lora(x, W, A, B, fine)
    y = ml.linear_lora(x, W, A, B, bad, workspace=ws)
    assert ml.debug_status(ws) == ml.FLAG_ADAPTER_RANGE
    assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 512, 100), (7, 512, 100), (40, 512, 100), (130, 512, 100), (520, 528, 203)])
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3")])
def test_linear_lora_strided_rows(T, K, N, act, w):
    """x, W, residual and y inside wider buffers, whose other columns hold NaN and stay untouched."""
    x, W, scale, b, r = _inputs(T, K, N, act, w, 11)
    A, B = _adapters(4, 16, K, W.shape[0], 11)
    ids = _ids(T, 4, "random")

    def inside(t, left, right):
        wide = torch.full((t.shape[0] + 1, left + t.shape[1] + right), float("nan") if t.dtype == BF else 127,
                          dtype=t.dtype, device=DEV)
        view = wide[:-1, left:left + t.shape[1]]
        view.copy_(t)
        return wide, view

    xw, xv = inside(x, 8, 24)
    Ww, Wv = inside(W, 16, 32)
    rw, rv = inside(r, 3, 2)
    yw, yv = inside(torch.zeros(T, N, dtype=BF, device=DEV), 5, 2)
    keep = yw.clone()
    out = ml.linear_lora(xv, Wv, A, B, ids, w_scale=scale, bias=b, act=act, residual=rv, y=yv)
    torch.cuda.synchronize()
    assert out is yv
    _compare(out, x, W, scale, b, act, r, A, B, ids)
    keep[:-1, 5:5 + N] = out
    assert torch.equal(torch.nan_to_num(keep, 9.0), torch.nan_to_num(yw, 9.0))
    # in place of the residual
    y = r.clone()
    assert ml.linear_lora(x, W, A, B, ids, w_scale=scale, bias=b, act=act, residual=y, y=y) is y
    assert torch.equal(y, out)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 64, 100, 600])
def test_linear_lora_poisoned_workspace_and_other_streams(T):
    K, N = 2048, 256
    x, W, _, b, r = _inputs(T, K, N, "swiglu", "bf16", 31)
    A, B = _adapters(5, 16, K, 2 * N, 31)
    ids = _ids(T, 5, "random")
    want = ml.linear_lora(x, W, A, B, ids, bias=b, act="swiglu", residual=r)
    d = ml.LinearLoraDims(ml.LinearDims(T, K, N, ml.ACTIVATIONS["swiglu"], 0, K, K, N, N), 5, 16)
    need = ml.lib().moe_lora_linear_lora_workspace_size(ctypes.byref(d))
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = ml.linear_lora(x, W, A, B, ids, bias=b, act="swiglu", residual=r, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert (ws[need:] == 255).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 64, 200])
def test_linear_lora_graph_replays(T):
    """Captured with a workspace of its own; other adapters at every replay, eager calls between."""
    K, N = 2048, 192
    x, W, _, b, r = _inputs(T, K, N, "swiglu", "bf16", 51)
    A, B = _adapters(9, 8, K, 2 * N, 51)
    ids = _ids(T, 9, "random")
    y = torch.empty(T, N, dtype=BF, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ml.linear_lora(x, W, A, B, ids, bias=b, act="swiglu", residual=r, y=y, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ml.linear_lora(x, W, A, B, ids, bias=b, act="swiglu", residual=r, y=y, workspace=ws)
    for i in range(4):
        x.copy_(torch.randn(T, K, device=DEV).to(BF))
        ids.copy_(_ids(T, 9, ["random", "distinct", "none", "one"][i], i))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ml.linear_lora(x, W, A, B, ids, bias=b, act="swiglu", residual=r)), i


@pytest.mark.gpu
def test_linear_lora_adapters_past_4_gib():
    """Byte offsets of the last adapter's A and B past 32 bits."""
    K, N, r, nA = 4096, 4096, 64, 8200  # 4.3 GB each
    A = torch.zeros(nA, r, K, dtype=BF, device=DEV)
    B = torch.zeros(nA, N, r, dtype=BF, device=DEV)
    small = _adapters(1, r, K, N, 3)
    A[-1], B[-1] = small[0][0], small[1][0]
    for T in (20, 100):
        x, W, _, _, _ = _inputs(T, K, N, "none", "bf16", T)
        ids = torch.where(torch.arange(T, device=DEV) % 3 == 0, nA - 1, 5).int()
        y = ml.linear_lora(x, W, A, B, ids)
        _compare(y, x, W, None, None, "none", None, small[0], small[1], torch.where(ids == nA - 1, 0, -1).int())


@pytest.mark.gpu
def test_linear_lora_from_two_threads():
    """Two threads, each on a stream of its own: the same bits as alone."""
    cases = []
    for T, K, N, act in ((50, 2048, 200, "swiglu"), (100, 2064, 131, "silu"), (300, 1040, 515, "none")):
        x, W, _, b, r = _inputs(T, K, N, act, "bf16", T)
        cases.append((x, W, *_adapters(6, 16, K, W.shape[0], T), _ids(T, 6, "random"), b, act, r))

    def calls():
        return [ml.linear_lora(x, W, A, B, ids, bias=b, act=act, residual=r) for x, W, A, B, ids, b, act, r in cases]

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
def test_linear_lora_empty_batch():
    W = torch.zeros(24, 16, dtype=BF, device=DEV)
    A, B = torch.zeros(1, 8, 16, dtype=BF, device=DEV), torch.zeros(1, 24, 8, dtype=BF, device=DEV)
    y = ml.linear_lora(torch.empty(0, 16, dtype=BF, device=DEV), W, A, B, torch.empty(0, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 24)


@pytest.mark.gpu
def test_linear_lora_refuses_tensors():
    T, K, N = 4, 64, 32
    x, W, _, _, r = _inputs(T, K, N, "none", "bf16", 1)
    A, B = _adapters(2, 8, K, N, 1)
    ids = _ids(T, 2, "random")
    good = dict(x=x, W=W, A=A, B=B, adapter_ids=ids)
    for name, bad in [("A", A[:, :, :32]), ("A", A.float()), ("A", A.transpose(0, 1)), ("B", B[:, :16]), ("B", B.half()),
                      ("B", None), ("A", None), ("adapter_ids", ids.long()), ("adapter_ids", ids[:2]), ("adapter_ids", None),
                      ("adapter_ids", ids.cpu()), ("A", A.cpu())]:
        with pytest.raises((TypeError, ValueError)):
            ml.linear_lora(**{**good, name: bad})
    with pytest.raises(ml.MoeLoraError):  # a rank of 12
        ml.linear_lora(x, W, torch.zeros(2, 12, K, dtype=BF, device=DEV), torch.zeros(2, N, 12, dtype=BF, device=DEV), ids)
    with pytest.raises(ValueError):
        ml.linear_lora(**good, y=B.view(-1)[:T * N].view(T, N))
    with pytest.raises(ValueError):
        ml.linear_lora(**good, y=r, workspace=A.view(-1).view(torch.uint8))
    with pytest.raises(ml.MoeLoraError):
        ml.linear_lora(**good, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_linear_lora_host_checks():
    lib = ml.lib()
    d = ml.LinearLoraDims(ml.LinearDims(4, 64, 32, 0, 0, 64, 64, 32, 32), 2, 8)
    need = lib.moe_lora_linear_lora_workspace_size(ctypes.byref(d))
    assert need > 0 and need % 256 == 0
    p = [0x10000 * (i + 1) for i in range(10)]

    def call(dims=d, ws=need, **change):
        q = dict(x=p[0], W=p[1], s=None, b=None, r=None, A=p[2], B=p[3], ids=p[4], y=p[5], w=p[6])
        q.update(change)
        return lib.moe_lora_linear_lora(q["x"], q["W"], q["s"], q["b"], q["r"], q["A"], q["B"], q["ids"],
                                        ctypes.byref(dims) if dims else None, q["y"], q["w"], ws, None)

    for name in ("x", "W", "A", "B", "ids", "y", "w"):
        assert call(**{name: None}) == ml.ENULL, name
    for name in ("x", "W", "A", "B"):
        assert call(**{name: p[0] + 8}) == ml.EALIGN, name
    for name, off in (("ids", 2), ("y", 1), ("b", 1), ("r", 1)):
        assert call(**{name: p[0] + off}) == ml.EALIGN, name
    assert call(s=p[7]) == ml.EUNSUPPORTED
    assert call(ws=need - 1) == ml.EWORKSPACE and call(w=p[6] + 16) == ml.EWORKSPACE
    assert call(dims=None) == ml.ENULL
    for field, values in (("rank", (0, 4, 12, 128, -8)), ("n_adapters", (0, -1, 1 << 28))):
        for v in values:
            b = ml.LinearLoraDims.from_buffer_copy(d)
            setattr(b, field, v)
            assert call(b) == ml.EINVAL_DIMS and lib.moe_lora_linear_lora_workspace_size(ctypes.byref(b)) == 0
    for field, v in (("T", 1 << 24), ("T", -1), ("in_features", 63), ("out_features", 0), ("act", 9), ("w_type", 7),
                     ("x_stride", 8), ("w_stride", 1 << 40)):
        b = ml.LinearLoraDims.from_buffer_copy(d)
        setattr(b.linear, field, v)
        assert call(b) == ml.EINVAL_DIMS, field
    b = ml.LinearLoraDims.from_buffer_copy(d)
    b.linear.T = 0
    assert call(b, x=None, W=None, A=None, B=None, ids=None, y=None, w=None) == ml.OK
    with pytest.raises(ValueError):
        ml.linear_lora(None, None, None, None, None, act="tanh")
    with pytest.raises(ml.MoeLoraError):
        ml.linear_lora_plan(4, 64, 32, 2, 12)


def _compare_broken(y, ref, bound):
    """Finite elements within the bound; infinities and NaNs where the formula has them, with their signs."""
    fin = torch.isfinite(ref)
    got, want = y.double()[~fin], ref[~fin]
    assert ((got == want) | (torch.isnan(got) & torch.isnan(want))).all(), \
        f"{int((got != want).sum() - (torch.isnan(got) & torch.isnan(want)).sum())} of {got.numel()}"
    assert torch.isfinite(y[fin]).all() and ((y.double() - ref).abs() <= bound)[fin].all()


def _broken_adapters(T, K, N, act, w, r, pattern):
    """An infinity in one adapter's A, infinities of both signs in another's B: the formula's results, and the same
    bits for every token without them."""
    print("linear_lora broken", T, K, N, act, w, r, pattern, flush=True)
    x, W, scale, _, res = _inputs(T, K, N, act, w, T + N + r, False, True)
    rows = W.shape[0]
    A, B = _adapters(3, r, K, rows, r)
    ids = _ids(T, 3, pattern, 3)
    want = ml.linear_lora(x, W, A, B, ids, w_scale=scale, act=act, residual=res)
    A[1, r // 2, 7] = math.inf
    B[2, min(5, rows - 1), 1] = math.inf
    B[2, rows // 2, r - 1] = -math.inf
    B[2, rows - 1, 0], B[2, rows - 1, 5] = math.inf, -math.inf
    y = ml.linear_lora(x, W, A, B, ids, w_scale=scale, act=act, residual=res)
    torch.cuda.synchronize()
    keep = (ids != 1) & (ids != 2)
    assert torch.equal(y[keep], want[keep])
    ref, bound = _reference(x, W, scale, None, act, res, A, B, ids)
    assert not torch.isfinite(ref[ids == 1]).any() and not torch.isfinite(ref[ids == 2][:, -1]).any()
    _compare_broken(y, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 256, 40), (1, 8192, 40), (2, 256, 64), (17, 272, 33), (30, 256, 64), (40, 512, 2000),
                                   (48, 272, 1040)])
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3")])
@pytest.mark.parametrize("r,pattern", [(8, "random"), (8, "one"), (16, "one"), (32, "random"), (64, "distinct")])
def test_linear_lora_infinite_adapters_of_few_tokens(T, K, N, act, w, r, pattern):
    """One token in one launch and in two; weights streamed for 16, 32 and 64 tokens, and small tiles."""
    assert ml.linear_lora_plan(T, K, N, 3, r, act, w == "e4m3")["streamed"] or (K, act) in ((8192, "none"), (8192, "swiglu"), (256, "swiglu"))
    _broken_adapters(T, K, N, act, w, r, pattern)


@pytest.mark.gpu
@pytest.mark.parametrize("r,pattern", [(8, "random"), (16, "one"), (32, "runs"), (64, "random")])
@pytest.mark.parametrize("act,w", [("none", "bf16"), ("swiglu", "bf16"), ("none", "e4m3")])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_linear_lora_infinite_adapters_of_every_form(form, act, w, r, pattern):
    """Every tile, with and without splits: groups of 32 tokens with one adapter, with some, and with none."""
    T, K, N, rows, cols, split = (SWIGLU_FORMS if act == "swiglu" else FORMS)[form]
    p = ml.linear_lora_plan(T, K, N, 3, r, act, w == "e4m3")
    assert (p["streamed"], p["tile_rows"], p["tile_cols"], p["splits"] > 1) == (0, rows, cols, split)
    _broken_adapters(T, K, N, act, w, r, pattern)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 8, 9, 32, 40, 512])
@pytest.mark.parametrize("nA,K", [(1, 2048), (40, 1024), (300, 4096), (512, 2048), (513, 4096), (1025, 528)])
@pytest.mark.parametrize("r", [8, 64])
def test_linear_lora_many_adapters_known(T, nA, K, r):
    """Few tokens of many adapters, on both sides of the borders between the shrink's forms and their splits."""
    _check(T, K, 48, "none", "bf16", r, nA, "random")
    if T > 1:
        _check(T, K, 48, "none", "bf16", r, nA, "distinct", seed=3)
