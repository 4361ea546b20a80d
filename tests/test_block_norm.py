"""The norms around a block (moe_lora_block_norm) against float64. Bounds: a sum over a row has at most 60
additions behind any of its terms (32 in a thread, 6 across a wavefront, 16 across the wavefronts; 2^-24 of the
sum of magnitudes each), every further operation 2^-24 of its result (exponential and reciprocals 2^-22), and each
output half a bf16 step; they are carried through the formulas in _reference."""
import ctypes
import math

import pytest
import torch

import lora_mixture_experts_amd as ml

DEV = "cuda"
BF = torch.bfloat16
U = 2.0 ** -24
SUM = 60 * U


def _norm(v, dv, w, b, layer, eps):
    """(norm, its error) of float64 rows v known within dv."""
    centre, dc = 0.0, 0.0
    if layer:
        centre = v.mean(1, keepdim=True)
        dc = dv.mean(1, keepdim=True) + (SUM + 2 * U) * v.abs().mean(1, keepdim=True)
    d = v - centre
    dd = dv + dc + U * d.abs()
    var = (d * d).mean(1, keepdim=True)
    dvar = (2 * d.abs() * dd + dd * dd).mean(1, keepdim=True) + (SUM + 3 * U) * var
    scale = 1 / (var + eps).sqrt()
    dscale = scale * (0.5 * dvar / (var + eps - dvar).clamp_min(1e-300) + 8 * U)
    wd = w.double()
    y = d * scale * wd
    dy = wd.abs() * (dd * scale + d.abs() * dscale + dd * dscale) + 3 * U * y.abs()
    if b is not None:
        y = y + b.double()
        dy = dy + U * y.abs()
    return y, dy


def _reference(y, residual, weight, bias, post_weight, post_bias, gate, sigmoid, rs, bs, norm, eps):
    layer = norm == "layer"
    r = residual.double()
    total, dt = rs * r, U * (rs * r).abs()
    if y is not None:
        b, db = y.double(), torch.zeros_like(r)
        if post_weight is not None:
            b, db = _norm(b, db, post_weight, post_bias, layer, eps)
        if gate is not None:
            g = gate.double()[:, None] if gate.dim() == 1 else gate.double()
            if sigmoid:
                g = torch.sigmoid(g)
                db = db + 2.0 ** -20 * b.abs()
            b, db = b * g, db * g.abs()
        total = total + bs * b
        dt = dt + abs(bs) * db + 4 * U * (bs * b).abs() + U * total.abs()
    out = None
    if weight is not None:
        out = _norm(total, dt, weight, bias, layer, eps)
    return (total, dt), out


def _within(got, pair):
    ref, d = pair
    assert torch.isfinite(got).all()
    bound = d + 2.0 ** -8 * (ref.abs() + d) + 2.0 ** -126
    worst = ((got.double() - ref).abs() / bound).max().item()
    assert worst <= 1.0, worst


def _inputs(T, h, post, gate, norm, seed=0, biases=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 31 * T + h)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    vec = lambda: (1 + 0.3 * normal(h)).to(BF)  # noqa: E731
    s = dict(y=normal(T, h).to(BF), residual=(2 * normal(T, h) + 0.5).to(BF), weight=vec(),
             bias=vec() if biases else None, post_weight=vec() if post else None,
             post_bias=vec() if post and biases else None, gate=None, sigmoid_gate=False)
    if gate in ("token", "sigmoid"):
        s["gate"], s["sigmoid_gate"] = 2 * normal(T), gate == "sigmoid"
    elif gate == "feature":
        s["gate"] = normal(1, h).to(BF).expand(T, h)
    elif gate == "element":
        s["gate"] = normal(T, h).to(BF)
    return s


def _call(s, norm, rs=0.75, bs=-1.5, eps=1e-5, **more):
    return ml.block_norm(**s, residual_scale=rs, branch_scale=bs, norm=norm, eps=eps, **more)


def _expect(s, norm, rs=0.75, bs=-1.5, eps=1e-5):
    return _reference(s["y"], s["residual"], s["weight"], s["bias"], s["post_weight"], s["post_bias"], s["gate"],
                      s["sigmoid_gate"], rs, bs, norm, eps)


SHAPES = [(1, 1), (3, 2), (1, 7), (5, 8), (2, 63), (9, 128), (4, 511), (3, 512), (2, 513), (7, 2040), (5, 2048), (3, 2049),
          (1, 4096), (6, 4099), (2, 8192), (3, 8193), (2, 16384), (2, 16391), (1, 32767), (2, 32768), (1000, 300),
          (700, 4100)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,h", SHAPES)
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post,gate", [(False, None), (True, "sigmoid"), (True, "feature")])
def test_block_norm_matches_float64(T, h, norm, post, gate):
    print("block_norm", T, h, norm, post, gate, flush=True)
    s = _inputs(T, h, post, gate, norm)
    total, out = _call(s, norm)
    torch.cuda.synchronize()
    want = _expect(s, norm)
    _within(total, want[0])
    _within(out, want[1])
    again = _call(s, norm)
    assert torch.equal(total, again[0]) and torch.equal(out, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [None, "token", "sigmoid", "feature", "element"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("biases", [False, True])
def test_block_norm_gates(gate, post, biases):
    s = _inputs(37, 777, post, gate, "rms", 3, biases)
    total, out = _call(s, "rms")
    want = _expect(s, "rms")
    _within(total, want[0])
    _within(out, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("h", [96, 1000, 4096])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_block_norm_one_side_only(h, norm):
    """Without a branch the norm alone; without a second norm the sum alone."""
    s = _inputs(11, h, False, None, norm, 5)
    total, out = ml.block_norm(None, s["residual"], s["weight"], bias=s["bias"], norm=norm)
    assert total is None
    _within(out, _reference(None, s["residual"], s["weight"], s["bias"], None, None, None, False, 1.0, 1.0, norm, 1e-6)[1])
    kept = torch.empty_like(out)
    total, _ = ml.block_norm(None, s["residual"], s["weight"], norm=norm, total=kept)
    assert total is kept and torch.equal(kept, s["residual"])
    total, out = ml.block_norm(s["y"], s["residual"])
    assert out is None
    _within(total, _reference(s["y"], s["residual"], None, None, None, None, None, False, 1.0, 1.0, norm, 1e-6)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("T,h", [(5, 40), (9, 513), (3, 4097), (1, 300)])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_block_norm_strided_rows(T, h, off):
    """Rows inside wider buffers at any offset, whose other columns stay as they are."""
    s = _inputs(T, h, True, "element", "layer", 7)
    want = _call(s, "layer")

    def inside(t):
        wide = torch.full((T + 1, off + h + 5), float("nan"), dtype=BF, device=DEV)
        wide[:-1, off:off + h] = t
        return wide, wide[:-1, off:off + h]

    views = {n: inside(s[n]) for n in ("y", "residual", "gate")}
    outs = {n: inside(torch.zeros(T, h, dtype=BF, device=DEV)) for n in ("total", "out")}
    keep = {n: outs[n][0].clone() for n in outs}
    got = _call({**s, **{n: views[n][1] for n in views}}, "layer", **{n: outs[n][1] for n in outs})
    torch.cuda.synchronize()
    for g, w, n in zip(got, want, ("total", "out")):
        assert g is outs[n][1] and torch.equal(g, w)
        keep[n][:-1, off:off + h] = w
        assert torch.equal(torch.nan_to_num(keep[n], 9.0), torch.nan_to_num(outs[n][0], 9.0))


@pytest.mark.gpu
@pytest.mark.parametrize("T,h", [(6, 100), (5, 2048), (300, 4100)])
def test_block_norm_in_place(T, h):
    """The residual stream in place, the next block's input over what the last one gave."""
    s = _inputs(T, h, True, "sigmoid", "rms", 9)
    want = _call(s, "rms")
    for total, out in (("residual", "y"), ("y", "residual"), ("residual", None), (None, "y")):
        c = {**s, "y": s["y"].clone(), "residual": s["residual"].clone()}
        more = {n: c[v] for n, v in (("total", total), ("out", out)) if v}
        got = _call(c, "rms", **more)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_block_norm_rows_keep_to_themselves():
    """Zero rows, rows with infinities and NaN, gates that are far out: no other row changes."""
    s = _inputs(12, 600, True, "sigmoid", "rms", 11)
    want = _call(s, "rms")
    c = {**s, "y": s["y"].clone(), "residual": s["residual"].clone(), "gate": s["gate"].clone()}
    c["y"][1, 5] = math.inf
    c["residual"][2, 5] = math.nan
    c["y"][3], c["residual"][3] = 0, 0
    c["gate"][4], c["gate"][5] = -math.inf, math.inf
    total, out = _call(c, "rms")
    rows = [0, 6, 7, 8, 9, 10, 11]
    assert torch.equal(total[rows], want[0][rows]) and torch.equal(out[rows], want[1][rows])
    assert torch.isnan(out[2]).all() and torch.isnan(total[2, 5])
    zeros = {**s, "post_bias": None, "bias": None, "y": c["y"][3:4], "residual": c["residual"][3:4], "gate": s["gate"][3:4]}
    total, out = _call(zeros, "rms")
    assert (total == 0).all() and (out == 0).all()
    one = {n: (v[4:5] if n in ("y", "residual", "gate") else v) for n, v in c.items()}
    total, _ = _call(one, "rms", rs=1.0)
    assert torch.equal(total, s["residual"][4:5])  # a closed gate


@pytest.mark.gpu
@pytest.mark.parametrize("h", [64, 4096])
def test_block_norm_large_mean(h):
    """LayerNorm of rows far from zero: the deviations, not the squares' difference."""
    s = _inputs(8, h, False, None, "layer", 13)
    s["residual"] = (1000 + 8 * torch.randn(8, h, device=DEV)).to(BF)
    total, out = _call(s, "layer", rs=1.0)
    _within(out, _expect(s, "layer", rs=1.0)[1])


@pytest.mark.gpu
def test_block_norm_stream_and_graph():
    s = _inputs(50, 2048, True, "sigmoid", "rms", 17)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _call(s, "rms")
    torch.cuda.current_stream().wait_stream(side)
    want = _call(s, "rms")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    total, out = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(s, "rms", total=total, out=out)
    for _ in range(4):
        s["y"].copy_(torch.randn(50, 2048, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = _call(s, "rms")
        assert torch.equal(total, want[0]) and torch.equal(out, want[1])


@pytest.mark.gpu
def test_block_norm_rows_past_4_gib():
    """Row offsets past 32 bits."""
    T, h, step = 3, 512, (3 << 30) // 2
    wide = torch.zeros(2 * step + h, dtype=BF, device=DEV)
    res = torch.as_strided(wide, (T, h), (step, 1))
    s = _inputs(T, h, False, None, "rms", 19)
    res.copy_(s["residual"])
    want = _call(s, "rms")
    got = _call({**s, "residual": res}, "rms", total=res)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(res, want[0])


@pytest.mark.gpu
def test_block_norm_empty_batch():
    y = torch.empty(0, 64, dtype=BF, device=DEV)
    total, out = ml.block_norm(y, y, torch.ones(64, dtype=BF, device=DEV))
    assert total.shape == (0, 64) and out.shape == (0, 64)


@pytest.mark.gpu
def test_block_norm_refuses_tensors():
    s = _inputs(4, 64, False, None, "rms", 1)
    for name, bad in [("y", s["y"][:, :32]), ("y", s["y"].float()), ("residual", s["residual"].t()), ("weight", s["weight"][:3]),
                      ("weight", s["weight"].float()), ("gate", torch.zeros(4, dtype=BF, device=DEV)),
                      ("gate", torch.zeros(4, 64, device=DEV)), ("gate", torch.zeros(3, device=DEV)), ("y", s["y"].cpu()),
                      ("residual", s["residual"][0])]:
        with pytest.raises((TypeError, ValueError)):
            _call({**s, name: bad}, "rms")
    wide = torch.zeros(4 * 64 + 64, dtype=BF, device=DEV)
    both = torch.as_strided(wide, (4, 64), (64, 1)), torch.as_strided(wide, (4, 64), (64, 1), 64)
    for more in (dict(total=both[0], out=both[1]), dict(total=both[0], out=both[0])):
        with pytest.raises(ValueError):
            _call(s, "rms", **more)
    with pytest.raises(ValueError):  # shifted, not the residual itself
        _call({**s, "residual": both[0]}, "rms", total=both[1])
    with pytest.raises(ml.MoeLoraError):
        _call({**s, "y": None, "gate": torch.zeros(4, device=DEV)}, "rms")
    with pytest.raises(ml.MoeLoraError):
        _call(s, "rms", eps=-1.0)
    with pytest.raises(ml.MoeLoraError):
        _call(s, "rms", rs=math.inf)
    with pytest.raises(ml.MoeLoraError):  # nothing to write
        ml.block_norm(None, s["residual"])


def test_block_norm_host_checks():
    lib = ml.lib()
    good = ml.BlockNormDims(4, 64, 0, 0, 1e-6, 1.0, 1.0, 64, 64, 0, 64, 64)
    p = [0x10000 * (i + 1) for i in range(10)]

    def call(d=good, **change):
        q = dict(y=p[0], residual=p[1], gate=None, pw=None, pb=None, w=p[2], b=None, sum=p[3], out=p[4])
        q.update(change)
        return lib.moe_lora_block_norm(q["y"], q["residual"], q["gate"], q["pw"], q["pb"], q["w"], q["b"],
                                       ctypes.byref(d) if d else None, q["sum"], q["out"], None)

    def dims(**change):
        d = ml.BlockNormDims.from_buffer_copy(good)
        for n, v in change.items():
            setattr(d, n, v)
        return d

    assert call(None) == ml.ENULL and call(residual=None) == ml.ENULL
    assert call(w=None) == ml.ENULL and call(out=None) == ml.ENULL and call(w=None, out=None, sum=None) == ml.ENULL
    assert call(gate=p[5]) == ml.ENULL and call(dims(gate=1)) == ml.ENULL
    assert call(pb=p[5]) == ml.EUNSUPPORTED and call(w=None, out=None, b=p[5]) == ml.EUNSUPPORTED
    assert call(y=None, pw=p[5]) == ml.EUNSUPPORTED and call(dims(gate=2), y=None, gate=p[5]) == ml.EUNSUPPORTED
    for name in ("y", "residual", "w", "b", "pw", "sum", "out"):
        assert call(**{name: p[6] + 1}) == ml.EALIGN, name
    assert call(dims(gate=1), gate=p[5] + 2) == ml.EALIGN and call(dims(gate=3), gate=p[5] + 1) == ml.EALIGN
    for change in (dict(T=-1), dict(T=1 << 30), dict(hidden=0), dict(hidden=32769), dict(norm=2), dict(gate=4), dict(eps=-1e-9),
                   dict(eps=math.nan), dict(residual_scale=math.inf), dict(branch_scale=math.nan), dict(y_stride=63),
                   dict(residual_stride=1 << 40), dict(sum_stride=0), dict(out_stride=-64), dict(gate=3, gate_stride=5)):
        assert call(dims(**change), gate=p[5] if change.get("gate") == 3 else None) == ml.EINVAL_DIMS, change
    assert call(dims(T=0), y=None, residual=None, w=None, out=None, sum=None) == ml.OK
    with pytest.raises(ValueError):
        ml.block_norm(None, None, norm="batch")


@pytest.mark.gpu
def test_block_norm_refuses_a_sigmoid_of_features():
    """The sigmoid is of a value a token: a gate of [T][h] would go in as it is."""
    for gate in ("feature", "element"):
        s = _inputs(4, 64, False, gate, "rms", 1)
        for T in (4, 1):
            one = {n: v[:T] if n in ("y", "residual", "gate") else v for n, v in s.items()}
            with pytest.raises(ValueError):
                _call({**one, "sigmoid_gate": True}, "rms")
            _call(one, "rms")


@pytest.mark.gpu
@pytest.mark.parametrize("T,h", [(5, 96), (3, 700), (2, 4096), (2, 20000)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("size,eps", [(2.0 ** -73, 0.0), (2.0 ** -73, 1e-44), (2.0 ** -66, 1e-38), (2.0 ** -100, 0.0),
                                      (2.0 ** -41, 0.0), (2.0 ** -45, 1e-28)])
def test_block_norm_small_rows(T, h, norm, size, eps):
    """Rows whose squares leave fp32's normal numbers, where eps does not outweigh them: the formula's results, of the
    block's norm and of the stream's."""
    s = _inputs(T, h, True, None, norm, 21)
    s["y"], s["residual"] = (size * s["y"].float()).to(BF), (size * s["residual"].float()).to(BF)
    s["post_weight"], s["post_bias"] = (size * s["post_weight"].float()).to(BF), None
    total, out = _call(s, norm, rs=1.0, bs=0.5, eps=eps)
    # (the call's eps is fp32, which has 7 * 2^-149 = 9.81e-45 for 1e-44: 2% less)
    want = _expect(s, norm, rs=1.0, bs=0.5, eps=torch.tensor(eps, dtype=torch.float32).item())
    _within(total, want[0])
    _within(out, want[1])
