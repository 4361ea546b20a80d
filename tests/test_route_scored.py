"""Expert choice (moe_lora_route) against a float64 implementation in numpy: rounds of "the largest
choice value, then the lowest id". Ids and empty slots must be equal; weights are compared under
the rounding bound of `_weight_bound`."""
import ctypes
import math

import numpy as np
import pytest
import torch

import lora_mixture_experts_amd as ml

DEV = "cuda"


def _reference(logits, k, scoring="softmax", bias=None, n_groups=1, topk_groups=1, group_score="max",
               renormalize=True, scale=1.0, token_mask=None):
    lg = np.asarray(logits, np.float64)
    T, E = lg.shape
    ok = np.isfinite(lg)
    if token_mask is not None:
        ok &= np.asarray(token_mask, bool)[:, None]
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    S = E // n_groups
    for t in range(T):
        live = np.nonzero(ok[t])[0]
        if live.size == 0:
            continue
        l = lg[t, live]
        if scoring == "softmax":
            ex = np.exp(l - l.max())
            s = ex / ex.sum()
        else:
            s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        if bias is not None:
            c = s + np.asarray(bias, np.float64)[live]
        else:
            c = s if n_groups > 1 and group_score == "top2" else l
        choice = {int(e): v for e, v in zip(live, c) if np.isfinite(v)}
        logit = dict(zip(live.tolist(), l))
        score = dict(zip(live.tolist(), s))
        if topk_groups < n_groups:
            rank = []
            for g in range(n_groups):
                vals = sorted((v for e, v in choice.items() if e // S == g), reverse=True)
                if vals:
                    rank.append((-(sum(vals[:2]) if group_score == "top2" else vals[0]), g))
            kept = {g for _, g in sorted(rank)[:topk_groups]}
            choice = {e: v for e, v in choice.items() if e // S in kept}
        best = sorted(choice, key=lambda e: (-choice[e], e))[:k]
        if not best:
            continue
        if renormalize:
            if scoring == "softmax":
                u = np.exp(np.array([logit[e] for e in best]) - max(logit[e] for e in best))
            else:  # over the largest common factor: scores that underflow keep their ratios
                lo = np.minimum([logit[e] for e in best], 0.0)
                u = np.exp(lo - lo.max()) / (1 + np.exp(-np.abs([logit[e] for e in best])))
            u = u / u.sum()
        else:
            u = np.array([score[e] for e in best])
        ids[t, :len(best)] = best
        w[t, :len(best)] = scale * u
    return ids, w


def _weight_bound(logits, k, w):
    """Relative error of a weight in units of 2^-23: an exponential and its sum's terms 4 each, the
    rounding of its argument (half a unit of it) twice, the sum over up to 38 partial sums, the
    division and the scaling; results under 2^-126 may be flushed."""
    fin = np.isfinite(logits)
    span = np.maximum(np.where(fin, logits, -np.inf).max(1) - np.where(fin, logits, np.inf).min(1), 0.0)
    return np.abs(w) * ((38 + 12 + np.minimum(span, 200.0))[:, None] * 2.0 ** -23) + 2.0 ** -125


def _check(logits, k, ids_bias=None, mask=None, **kw):
    print("route", tuple(logits.shape), k, {a: b for a, b in kw.items()}, flush=True)
    flags = torch.full((logits.shape[0],), 7, dtype=torch.int32, device=DEV)
    ids, w = ml.route(logits.to(DEV) if not logits.is_cuda else logits, k,
                      bias=None if ids_bias is None else ids_bias.to(DEV),
                      token_mask=None if mask is None else mask.to(DEV), token_flags=flags, **kw)
    torch.cuda.synchronize()
    lg = logits.cpu().numpy()
    rid, rw = _reference(lg, k, bias=None if ids_bias is None else ids_bias.numpy(),
                         token_mask=None if mask is None else mask.numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    err = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert np.all(err <= _weight_bound(lg, k, rw)), float((err - _weight_bound(lg, k, rw)).max())
    want = (~np.isfinite(lg)).any(1)
    if mask is not None:
        want &= mask.numpy()
    np.testing.assert_array_equal(flags.cpu().numpy(), want.astype(np.int32))
    return ids, w


def _logits(T, E, seed, spread=1.0):
    return spread * torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32))


SHAPES = [
    # T, E, k, groups, kept groups
    (1, 1, 1, 1, 1), (1, 16, 2, 1, 1), (3, 5, 5, 1, 1), (64, 64, 6, 1, 1), (70, 128, 8, 8, 3), (33, 256, 8, 8, 4),
    (9, 160, 6, 5, 3), (5, 1024, 16, 1, 1), (6, 1000, 13, 4, 2), (4, 1023, 11, 33, 7), (5, 192, 8, 64, 9),
    (7, 36, 3, 12, 4), (2051, 16, 2, 1, 1), (2500, 60, 4, 3, 2), (2100, 256, 8, 8, 4), (2049, 129, 16, 1, 1),
    (2300, 64, 1, 16, 2), (2200, 40, 7, 5, 2), (2100, 250, 9, 2, 1), (2060, 512, 8, 8, 4), (2050, 6, 2, 1, 1),
    (3000, 144, 12, 16, 5),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
@pytest.mark.parametrize("scoring,group_score,renorm,biased", [
    ("softmax", "max", True, False), ("softmax", "top2", False, True), ("sigmoid", "top2", True, True),
    ("sigmoid", "max", False, False), ("sigmoid", "top2", True, False), ("softmax", "max", False, False)])
def test_route_matches_float64(T, E, k, G, tg, scoring, group_score, renorm, biased):
    L = _logits(T, E, T + E + k)
    bias = 0.2 * _logits(1, E, 5)[0] if biased else None
    _check(L, k, bias, scoring=scoring, n_groups=G, topk_groups=tg, group_score=group_score, renormalize=renorm,
           scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [50, 2100])
@pytest.mark.parametrize("E,k,G,tg", [(16, 4, 1, 1), (128, 8, 4, 2), (60, 5, 5, 2), (256, 16, 8, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_id(T, E, k, G, tg, scoring):
    """Few levels: most comparisons are ties, of experts and of groups; +0 and -0 tie too."""
    rng = np.random.default_rng(E)
    L = np.round(rng.standard_normal((T, E))).astype(np.float32)
    L[L == 0] = np.where(rng.random(int((L == 0).sum())) < 0.5, -0.0, 0.0)
    L = torch.from_numpy(L)
    _check(L, k, scoring=scoring, n_groups=G, topk_groups=tg)
    bias = torch.from_numpy(np.round(2 * rng.standard_normal(E)).astype(np.float32) / 4)
    _check(L, k, bias, scoring=scoring, n_groups=G, topk_groups=tg)
    _check(L, k, torch.zeros(E), scoring=scoring, n_groups=G, topk_groups=tg)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 2200])
@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_masked_experts_and_rows(T, scoring, biased):
    """-inf, +inf and NaN logits are never chosen, whatever the bias; a token with fewer experts
    than slots leaves the rest empty, one without any all of them; padded rows are not read."""
    E, k, G = 48, 6, 4
    rng = np.random.default_rng(T)
    L = _logits(T, E, 3)
    drop = rng.random((T, E)) < rng.choice([0.1, 0.9, 1.0], T)[:, None]
    L[torch.from_numpy(drop)] = -math.inf
    L[0] = math.nan
    L[1, :47] = math.nan
    L[2] = math.inf
    L[3, ::2] = math.inf
    mask = torch.from_numpy(rng.random(T) < 0.7)
    L[torch.from_numpy(~mask.numpy())] = math.nan
    bias = 0.3 * _logits(1, E, 9)[0] if biased else None
    if biased:
        bias[5], bias[6], bias[7] = -math.inf, math.nan, math.inf
        bias[11] = 40.0
    _check(L, k, bias, scoring=scoring)
    _check(L, k, bias, mask, scoring=scoring, n_groups=G, topk_groups=2, group_score="top2")
    _check(L, k, bias, torch.zeros(T, dtype=torch.bool), scoring=scoring)


@pytest.mark.gpu
@pytest.mark.parametrize("spread,shift", [(30.0, 0.0), (1.0, 80.0), (1.0, -80.0), (5.0, -300.0), (1e-6, 0.0)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_far_logits(spread, shift, scoring):
    """Scores that saturate or underflow in fp32: order by logits, weights by their ratios."""
    L = _logits(65, 32, 17, spread) + shift
    _check(L, 4, scoring=scoring, renormalize=True)
    _check(L, 4, scoring=scoring, renormalize=False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 2100])
@pytest.mark.parametrize("E,k,G,tg", [(64, 8, 1, 1), (256, 8, 8, 4), (400, 16, 1, 1), (48, 5, 4, 1), (16, 2, 1, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_choices_closer_than_fp32(T, E, k, G, tg, scoring):
    """Biases that bring every choice value of one token to within an fp32 rounding (6e-8) of 0.7:
    neighbours, group sums and the last slot's border are told apart in double."""
    L = _logits(1, E, 23)
    l = L[0].double()
    s = torch.softmax(l, 0) if scoring == "softmax" else torch.sigmoid(l)
    bias = (0.7 - s).float()
    c = (s + bias.double()).numpy()
    gaps = np.diff(np.sort(c))
    assert gaps.max() < 1e-7 and np.median(gaps) > 2e-12  # (told apart by 2^-42 = 2.3e-13)
    rows = L.repeat(T, 1)
    if T > 2:
        rows[::2] = _logits((T + 1) // 2, E, 24)  # others beside it in the wavefront
    _check(rows, k, bias, scoring=scoring, n_groups=G, topk_groups=tg, group_score="top2")
    _check(rows, k, bias, scoring=scoring, n_groups=G, topk_groups=tg, group_score="max")


def _far_rows(T, E, shift):
    """By row, one of each to a wavefront of four: few levels around 0 (ties, which are settled in
    double), normal logits moved by `shift`, one level there, every third expert switched off there."""
    L = _logits(T, E, 29)
    L[::4] = torch.round(L[::4])
    L[1::4] += shift
    L[2::4] = shift
    L[3::4] += shift
    L[3::4, ::3] = -math.inf
    return L


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [-650.0, -700.0, -1000.0, -1500.0, -1e4, -1e9, 1e4])
@pytest.mark.parametrize("E,k,G,tg", [(32, 4, 8, 4), (256, 8, 8, 3), (96, 5, 1, 1)])
def test_route_far_logits_ranked_by_softmax_scores(shift, E, k, G, tg):
    """A softmax depends on the differences of the logits only, wherever they lie."""
    L = _far_rows(65, E, shift)
    bias = 0.02 * _logits(1, E, 31)[0]
    for b in (None, bias, torch.zeros(E)):
        for group_score in ("top2", "max"):
            _check(L, k, b, n_groups=G, topk_groups=tg, group_score=group_score, renormalize=False)
            _check(L, k, b, n_groups=G, topk_groups=tg, group_score=group_score)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,tg", [(32, 4, 8, 4), (256, 8, 8, 3), (96, 5, 1, 1)])
def test_route_rows_of_the_lowest_float(scoring, E, k, G, tg):
    """torch.finfo(float32).min is finite: a logit like any other, for a whole row, for a part of it
    and beside the largest float."""
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    L = _logits(65, E, 37)
    L[::4] = low
    L[1::4, : E // 2] = low
    L[2::4] = -math.inf
    L[2::4, 1::3] = low
    L[3, 1:] = low
    L[3, 0] = high
    L[7] = high
    bias = 0.02 * _logits(1, E, 41)[0]
    for b in (None, bias):
        for group_score in ("top2", "max"):
            for renorm in (True, False):
                kw = dict(scoring=scoring, n_groups=G, topk_groups=tg, group_score=group_score, renormalize=renorm)
                if scoring == "softmax":
                    _check(L, k, b, **kw)
                    continue
                # Two sigmoids of the lowest float are more than one: float64 cannot hold either, but both
                # at -700, where nothing else ranks below or between and the weights are still 0.
                ids, w = ml.route(L.to(DEV), k, bias=None if b is None else b.to(DEV), **kw)
                near = torch.where(L == low, -700.0, L).numpy()
                rid, rw = _reference(near, k, bias=None if b is None else b.numpy(), **kw)
                np.testing.assert_array_equal(ids.cpu().numpy(), rid)
                assert np.all(np.abs(w.cpu().numpy() - rw) <= _weight_bound(near, k, rw))


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [5, 4099])
def test_route_group_sums_whose_biases_cancel(scoring, T):
    """Two experts a group with biases 4096 and -4096: a group's score is the sum of its two scores,
    but a choice value in fp32 is off by up to 2^-12."""
    G, tg = 16, 5
    L = _logits(T, 2 * G, 43)
    bias = torch.tensor([4096.0, -4096.0]).repeat(G)
    l = L.double()
    s = (torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)).view(T, G, 2)
    for v in (s.sum(2), s[:, :, 0], s[:, :, 1]):  # (told apart by 2^-42 of 4096, 1e-9)
        assert v.sort(1).values.diff(dim=1).min() > 4e-9
    _check(L, tg, bias, scoring=scoring, n_groups=G, topk_groups=tg, group_score="top2")


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
def test_route_one_token_of_any_stride(bias):
    """The stride of a single row is never stepped: the last position of a long sequence, a view
    whose stride is less than its row."""
    E, k = 64, 6
    b = 0.1 * _logits(1, E, 47)[0] if bias else None
    long = torch.empty(1, 1 << 16, E, device=DEV)
    long[:, -1] = _logits(1, E, 53).to(DEV)
    assert long[:, -1].stride(0) >= 1 << 22
    _check(long[:, -1], k, b)
    _check(torch.as_strided(long, (1, E), (3, 1), ((1 << 16) - 1) * E), k, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [17, 2100])
def test_route_strided_and_unaligned_rows(T):
    wide = torch.randn(T, 77, device=DEV)
    _check(wide[:, 3:67], 8, n_groups=4, topk_groups=2)
    _check(wide[:, 4:68], 8, 0.1 * torch.randn(64), scoring="sigmoid")
    big = torch.randn(T, 256, device=DEV)
    bias = (0.1 * torch.randn(260)).to(DEV)[1:257]  # 4-byte aligned only
    ids, _ = ml.route(big, 8, scoring="sigmoid", bias=bias, n_groups=8, topk_groups=4, group_score="top2")
    ref, _ = _reference(big.cpu().numpy(), 8, "sigmoid", bias.cpu().numpy(), 8, 4, "top2")
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)


@pytest.mark.gpu
def test_route_writes_its_rows_only_and_runs_on_other_streams():
    T, E, k = 2053, 128, 8
    L = torch.randn(T, E, device=DEV)
    want = ml.route(L, k)
    ids = torch.full((T + 3, k), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 3, k), 7.5, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ml.route(L, k, topk_ids=ids[:T], topk_w=w[:T])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(ids[:T], want[0]) and torch.equal(w[:T], want[1])
    assert (ids[T:] == 77).all() and (w[T:] == 7.5).all()


@pytest.mark.gpu
def test_route_empty_batch():
    ids, w = ml.route(torch.empty(0, 8, device=DEV), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


# ----------------------------------------------------------------------------- refusals (CPU)

def _call(ptrs=None, **kw):
    f = dict(T=4, n_experts=16, topk=2, scoring=0, n_groups=1, topk_groups=1, group_score=0, renormalize=1,
             scale=1.0, logits_stride=16)
    f.update(kw)
    p = [0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000] if ptrs is None else ptrs
    r = ml.Router(**f)
    return ml.lib().moe_lora_route(p[0], p[1], p[2], ctypes.byref(r), p[3], p[4], p[5], None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 26), dict(n_experts=0), dict(n_experts=1025, logits_stride=1025), dict(topk=0), dict(topk=17),
    dict(n_experts=4, topk=5), dict(scoring=2), dict(scoring=-1), dict(n_groups=0), dict(n_groups=3),
    dict(n_experts=130, n_groups=65, topk_groups=65, logits_stride=130), dict(topk_groups=0),
    dict(n_groups=4, topk_groups=5), dict(n_groups=16, topk_groups=1), dict(group_score=2), dict(renormalize=2),
    dict(scale=math.inf), dict(scale=math.nan), dict(logits_stride=15), dict(logits_stride=1 << 22)])
def test_route_refuses_fields_out_of_range(bad):
    assert _call(**bad) == ml.EINVAL_DIMS


def test_route_refuses_more_tokens_than_a_launch_holds():
    """Four tokens a workgroup of 256 threads, fewer than 2^32 threads a launch."""
    odd = [0x10002, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000]  # (refused next, whatever the sizes)
    assert _call(odd, T=(1 << 26) - 4, n_experts=1024, logits_stride=1024) == ml.EALIGN
    for T in ((1 << 26) - 3, (1 << 26) - 1):
        assert _call(odd, T=T, n_experts=1024, logits_stride=1024) == ml.EINVAL_DIMS


def test_route_refuses_pointers():
    base = [0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000]
    for i in (0, 3, 4):
        p = list(base)
        p[i] = None
        assert _call(p) == ml.ENULL
    for i in (0, 1, 3, 4, 5):
        p = list(base)
        p[i] += 2
        assert _call(p) == ml.EALIGN
    assert ml.lib().moe_lora_route(*base[:3], None, *base[3:], None) == ml.ENULL
    assert _call([None] * 6, T=0) == ml.OK


def test_route_binding_refuses():
    with pytest.raises(ValueError):
        ml.route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        ml.route(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        ml.route(torch.zeros(8), 2)


@pytest.mark.gpu
def test_route_refuses_choices_before_it_allocates():
    logits = torch.randn(4, 32, device=DEV)
    for k in (33, 2 ** 31 - 1, 0, -1):
        with pytest.raises(ml.MoeLoraError):
            ml.route(logits, k)


@pytest.mark.gpu
def test_route_refuses_outputs_over_arguments():
    T, E, k = 6, 64, 4
    buf = torch.randn(T, 3 * E, device=DEV)
    logits, bias = buf[:, :E], torch.zeros(E + T * k, device=DEV)
    want = ml.route(logits, k)
    mask = torch.ones(4 * T + T, dtype=torch.uint8, device=DEV)
    bad = [dict(topk_w=buf.view(-1)[E - 1:E - 1 + T * k].view(T, k)), dict(topk_w=bias[E - 1:E - 1 + T * k].view(T, k)),
           dict(topk_ids=buf.view(torch.int32).view(-1)[:T * k].view(T, k)),
           dict(token_flags=buf.view(torch.int32).view(-1)[-2 * E - 1:-2 * E - 1 + T]),
           dict(token_flags=mask[:4 * T].view(torch.int32), token_mask=mask[4 * T - 1:5 * T - 1].view(torch.bool))]
    both = torch.zeros(T * k + 4, device=DEV)
    bad.append(dict(topk_w=both[:T * k].view(T, k), topk_ids=both.view(torch.int32)[4:].view(T, k)))
    bad.append(dict(topk_w=both[:T * k].view(T, k), token_flags=both.view(torch.int32)[:T]))
    for kw in bad:
        with pytest.raises(ValueError, match="overlaps"):
            ml.route(logits, k, bias=bias[:E], **kw)
    rest = torch.zeros(2 * T * k + T, dtype=torch.int32, device=DEV)  # side by side
    ids, w = ml.route(logits, k, bias=bias[:E], token_mask=mask[4 * T:].view(torch.bool),
                      topk_ids=rest[:T * k].view(T, k), topk_w=rest[T * k:2 * T * k].view(torch.float32).view(T, k),
                      token_flags=mask[:4 * T].view(torch.int32))
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
    ids, w = ml.route(logits, k, topk_w=buf.view(-1)[E:E + T * k].view(T, k))  # between two rows
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
