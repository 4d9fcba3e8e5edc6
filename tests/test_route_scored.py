"""Routing with scores (moe_mxfp4_route_scored): the oracle against brute force and the
refusals (CPU); ids, counts, offsets, perm and inv equal to the fp64 oracle's, and the
weights within the rounding of their fp32 evaluation (GPU)."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
import moe_expert_gemm_mxfp4_b200 as mx
from moe_expert_gemm_mxfp4_b200 import _lib

DEV = "cuda:0"
SCORES = {"softmax": mx.SCORE_SOFTMAX, "sigmoid": mx.SCORE_SIGMOID}


# ---------------------------------------------------------------- oracle

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_oracle_against_enumeration(score):
    """On few experts: the best set of groups, then of experts, by enumeration of all."""
    g = np.random.default_rng(0)
    E, G, tg, k = 8, 4, 2, 3
    for _ in range(20):
        l, b = g.normal(size=(1, E)), g.normal(size=E) * 0.1
        r = oracle.route_scored(l, k, score, b, G, tg, 2, True, 2.5)
        s = [1 / (1 + math.exp(-v)) for v in l[0]]
        if score == "softmax":
            s = [math.exp(v) / math.fsum(math.exp(u) for u in l[0]) for v in l[0]]
        c = [u + v for u, v in zip(s, b)]
        groups = max(itertools.combinations(range(G), tg),
                     key=lambda gs: math.fsum(c[2 * q] + c[2 * q + 1] for q in gs))
        allowed = [e for q in groups for e in (2 * q, 2 * q + 1)]
        best = max(itertools.combinations(allowed, k), key=lambda es: math.fsum(c[e] for e in es))
        assert set(r["ids"][0]) == set(best)
        assert list(r["ids"][0]) == sorted(best, key=lambda e: -c[e])
        assert np.allclose(r["w"][0], [2.5 * s[e] / math.fsum(s[q] for q in best) for e in r["ids"][0]], rtol=1e-12)


def test_oracle_renormalised_softmax_is_the_plain_routing():
    l = np.random.default_rng(1).normal(size=(50, 16)).astype(np.float32)
    a, b = oracle.route_scored(l, 4), oracle.route(l, 4)
    for key in ("ids", "counts", "offsets", "perm", "inv"):
        assert np.array_equal(a[key], b[key])
    assert np.allclose(a["w"], b["w"], rtol=1e-12)


# ---------------------------------------------------------------- refusals (CPU)

A, U, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001), ctypes.c_void_p(0)


def test_argument_checks():
    from moe_expert_gemm_mxfp4_b200 import build as mxbuild
    mxbuild.build()
    lib = _lib.load()

    def call(logits=A, dt=1, T=64, E=64, k=4, score=0, bias=N, G=8, tg=4, gt=2, scale=1.0, ids=A, perm=A, ws=A,
             nbytes=1 << 20):
        return lib.moe_mxfp4_route_scored(logits, dt, T, E, k, score, bias, G, tg, gt, 1, scale, ids, A, A, A, perm, A,
                                          ws, nbytes, N)

    inv, shape = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED_SHAPE
    for kw in (dict(logits=N), dict(ids=N), dict(perm=N), dict(T=0), dict(E=0), dict(k=0), dict(k=-1), dict(G=0),
               dict(tg=0), dict(dt=2), dict(score=2), dict(score=-1), dict(gt=0), dict(gt=3),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**kw) == inv, kw
    for kw in (dict(E=257, G=1, tg=1), dict(E=264, G=8), dict(k=9), dict(E=66, G=8), dict(G=64), dict(tg=9),
               dict(E=8, G=8, gt=2), dict(E=16, G=8, tg=1, k=3), dict(E=4, G=1, tg=1, k=5),
               dict(T=(1 << 31) // 4), dict(T=1 << 31, k=1), dict(T=1 << 62)):
        assert call(**kw) == shape, kw
    for kw in (dict(logits=U), dict(bias=U), dict(ids=U), dict(perm=U), dict(ws=U)):
        assert call(**kw) == _lib.ERR_MISALIGNED, kw
    need = mx.moe_mxfp4_route_scored_workspace_size(64, 64, 4)
    if need:
        assert call(nbytes=need - 1) == _lib.ERR_WORKSPACE
        assert call(ws=N, nbytes=0) == _lib.ERR_WORKSPACE
    big = mx.moe_mxfp4_route_scored_workspace_size(65536, 256, 8)
    assert big > 0 and call(T=65536, E=256, k=8, nbytes=big - 1) == _lib.ERR_WORKSPACE
    assert mx.moe_mxfp4_route_scored_workspace_size(0, 8, 2) == 0


def test_binding_refusals():
    f = mx.moe_mxfp4_route_scored
    z = torch.zeros(8, 32)
    with pytest.raises(ValueError, match="2-D"):
        f(torch.zeros(32), 4)
    with pytest.raises(ValueError, match="dtype"):
        f(z.double(), 4)
    with pytest.raises(ValueError, match="dtype"):
        f(z.half(), 4)
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(32, 8).t(), 4)
    with pytest.raises(ValueError, match="bias: expected dtype"):
        f(z, 4, bias=torch.zeros(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="bias: expected shape"):
        f(z, 4, bias=torch.zeros(31))
    with pytest.raises(ValueError, match="CUDA"):
        f(z, 4)


# ---------------------------------------------------------------- parity (GPU)

def _check(logits, k, bf16=False, **kw):
    logits = logits.to(torch.bfloat16) if bf16 else logits.float()
    bias = kw.get("bias")
    dev = dict(kw, score=SCORES[kw.get("score", "softmax")], bias=None if bias is None else bias.to(DEV))
    r = mx.moe_mxfp4_route_scored(logits.to(DEV), k, **dev)
    torch.cuda.synchronize()
    l = logits.double().numpy()
    ref = oracle.route_scored(l, k, **dict(kw, bias=None if bias is None else bias.double().numpy()))
    for key in ("ids", "counts", "offsets", "perm", "inv"):
        assert np.array_equal(r[key].cpu().numpy(), ref[key]), key
    w, want = r["weights"].cpu().numpy().astype(np.float64), ref["w"]
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(w), nan)
    # fp32 evaluation of the weights: the exponent's argument d = l - m is rounded (|d| 2^-24
    # of the result), exp is off by at most 2 ulp (2^-22), each of the at most 13 additions of a
    # sum, the quotients and the scale by 2^-24 more; so (|d| + 32) 2^-24 of the weight
    fin = np.where(np.isfinite(l), l, 0.0)
    d = (fin.max(1) - fin.min(1))[:, None] + np.abs(fin).max(1)[:, None]
    tol = (d + 32) * 2.0 ** -24 * np.abs(want) + 2.0 ** -126
    assert np.all((np.abs(w - want) <= tol)[~nan]), np.nanmax(np.abs(w - want) / np.maximum(np.abs(want), 1e-30))
    return r


def _logits(T, E, seed, scale=1.5):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * scale


def _bias(E, seed, scale=0.05):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed + 999)) * scale


# token counts on both sides of a warp round, of one chunk and of the chunk limit; expert
# counts off every multiple; every number of lanes per group
@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,tg,gt", [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (2, 3, 2, 3, 2, 1), (16, 32, 4, 1, 1, 1), (17, 33, 5, 1, 1, 1),
    (33, 34, 6, 17, 4, 2), (64, 256, 8, 8, 4, 2), (100, 60, 7, 5, 3, 2), (128, 96, 6, 6, 3, 2), (129, 255, 8, 17, 9, 1),
    (333, 96, 8, 32, 8, 1), (500, 64, 1, 4, 1, 2), (512, 256, 8, 32, 3, 2), (513, 254, 8, 2, 1, 2),
    (2367, 90, 6, 6, 3, 1), (2369, 72, 3, 9, 2, 2), (5000, 256, 8, 16, 5, 2)])
def test_against_oracle(score, T, E, k, G, tg, gt):
    for i, (bias, renorm, scale, bf16) in enumerate([(True, True, 2.5, False), (False, False, 1.0, True),
                                                     (True, False, 1.0, True)]):
        _check(_logits(T, E, T + E + i), k, bf16=bf16, score=score, bias=_bias(E, T + i) if bias else None,
               n_groups=G, top_groups=tg, group_top=gt, renorm=renorm, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gt", [1, 2])
def test_ties_masks_infinities_and_nan(score, gt):
    E, G, k = 48, 6, 5
    l = _logits(64, E, 3)
    inf, nan = float("inf"), float("nan")
    l[0] = 0.0                          # every expert alike
    l[1] = -inf                         # nothing left
    l[2] = -inf
    l[2, 20] = 0.5                      # one expert left
    l[3, 8:] = -inf                     # one group left
    l[4, ::2] = nan
    l[5] = nan
    l[6, 7] = inf
    l[7, [3, 40]] = inf
    l[8, 5], l[8, 6] = nan, -inf
    l[9] = -3e38
    l[10] = 3e38
    l[11] = 90.0
    l[12] = -95.0 + torch.arange(E) * 1e-3   # sigmoid scores near the smallest numbers
    l[13] = torch.arange(E) % 3         # many exact ties
    l[14, :40] = -inf
    l[15] = -0.0
    l[15, ::3] = 0.0
    for bias in (None, torch.zeros(E), _bias(E, 5)):
        for renorm in (True, False):
            _check(l, k, score=score, bias=bias, n_groups=G, top_groups=2, group_top=gt, renorm=renorm)
            _check(l, k, score=score, bias=bias, renorm=renorm)
    b = _bias(E, 6)
    b[3], b[4], b[5] = inf, -inf, nan
    _check(l, k, score=score, bias=b, n_groups=G, top_groups=3, group_top=gt)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_a_rounding_apart_are_not_swapped(score):
    """Choice values whose order only 64 bits show: neighbouring fp32 logits, and biases
    that undo the scores' differences to the last bits."""
    T, E, k = 256, 64, 8
    l = _logits(T, E, 11)
    bits = l[:, 0].view(torch.int32)
    for e in range(1, 12):              # a run of adjacent floats
        l[:, e] = (bits + e % 5).view(torch.float32)
    _check(l, k, score=score)
    l[:] = l[:1]                        # one row of scores s; bias ~ 0.5 - s leaves c near 0.5
    x = l[0].double()
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 0)
    bias = (0.5 - p).float()
    _check(l, k, score=score, bias=bias)
    _check(l, k, score=score, bias=bias, n_groups=8, top_groups=3, group_top=2)


@pytest.mark.gpu
def test_own_stream_and_graph():
    T, E, k = 3000, 128, 4
    l, b = _logits(T, E, 21).to(DEV), _bias(E, 22).to(DEV)
    kw = dict(score=mx.SCORE_SIGMOID, bias=b, n_groups=4, top_groups=2, group_top=2)
    want = mx.moe_mxfp4_route_scored(l, k, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.moe_mxfp4_route_scored(l, k, stream=side, **kw)
    side.synchronize()
    for key in want:
        assert torch.equal(got[key], want[key])
    buf = l.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = mx.moe_mxfp4_route_scored(buf, k, **kw)
    buf.copy_(_logits(T, E, 23))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    ref = oracle.route_scored(buf.double().cpu().numpy(), k, "sigmoid", b.double().cpu().numpy(), 4, 2, 2)
    for key in ("ids", "counts", "offsets", "perm", "inv"):
        assert np.array_equal(cap[key].cpu().numpy(), ref[key])


@pytest.mark.gpu
def test_workspace_and_outputs_stay_inside():
    from test_guard_gpu import Guarded
    T, E, k = 777, 90, 6
    l = _logits(T, E, 31).to(DEV)
    out = dict(ids=Guarded((T, k), torch.int32), weights=Guarded((T, k), torch.float32), counts=Guarded((E,), torch.int32),
               offsets=Guarded((E + 1,), torch.int32), perm=Guarded((T * k,), torch.int32), inv=Guarded((T * k,), torch.int32))
    need = mx.moe_mxfp4_route_scored_workspace_size(T, E, k)
    ws = Guarded((max(need, 16),), torch.uint8)
    p = {n: ctypes.c_void_p(g.t.data_ptr()) for n, g in out.items()}
    st = _lib.load().moe_mxfp4_route_scored(ctypes.c_void_p(l.data_ptr()), _lib.IN_F32, T, E, k, 1, N, 6, 2, 2, 1, 1.0,
                                            p["ids"], p["weights"], p["counts"], p["offsets"], p["perm"], p["inv"],
                                            ctypes.c_void_p(ws.t.data_ptr()), need, N)
    assert st == 0
    for n, g in out.items():
        g.check(n)
    ws.check("workspace")
    ref = oracle.route_scored(l.double().cpu().numpy(), k, "sigmoid", None, 6, 2, 2)
    assert np.array_equal(out["inv"].t.cpu().numpy(), ref["inv"])


# past one round of warps two tokens share a warp: odd last tokens, every number of lanes per group, groups
# that half a warp does not hold (3 of 85), more groups than half a warp has lanes
@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,tg,gt", [
    (4736, 32, 4, 1, 1, 1), (4737, 32, 4, 1, 1, 1), (4801, 90, 6, 6, 3, 1), (5003, 256, 8, 8, 4, 2), (4999, 255, 7, 3, 2, 2),
    (9475, 16, 8, 16, 9, 1), (5001, 64, 8, 32, 8, 2), (6007, 1, 1, 1, 1, 1), (5555, 200, 8, 1, 1, 1)])
def test_many_tokens_against_oracle(T, E, k, G, tg, gt):
    for i, (score, bias, renorm, bf16) in enumerate([("softmax", False, True, True), ("sigmoid", True, True, False),
                                                     ("softmax", True, False, False), ("softmax", False, True, False)]):
        _check(_logits(T, E, T + E + i), k, bf16=bf16, score=score, bias=_bias(E, T + i) if bias else None,
               n_groups=G, top_groups=tg, group_top=gt, renorm=renorm)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_that_share_a_warp_do_not_mix(score):
    """Rows that take the slow paths (ties, masks, infinities, NaN, long runs of near values) beside
    ordinary ones and beside each other, in both halves."""
    T, E, G, k = 4999, 48, 6, 5
    l = _logits(T, E, 41)
    inf, nan = float("inf"), float("nan")
    odd = torch.zeros(10, E)
    odd[1] = -inf
    odd[2, ::2] = nan
    odd[3, 7] = inf
    odd[4] = -3e38
    odd[5] = torch.arange(E) % 3
    odd[6, 8:] = -inf
    odd[7] = 1.0 + torch.arange(E) * 2.0 ** -23
    odd[8, :20] = -inf
    odd[9] = 90.0
    g = torch.Generator().manual_seed(42)
    at = torch.randperm(T, generator=g)[:1500]
    l[at] = odd[torch.randint(10, (1500,), generator=g)]
    l[T - 1] = odd[5]
    for bias in (None, _bias(E, 43)):
        for kw in (dict(), dict(n_groups=G, top_groups=2, group_top=2), dict(n_groups=G, top_groups=3, renorm=False)):
            _check(l, k, score=score, bias=bias, **kw)
            _check(l, k, bf16=True, score=score, bias=bias, **kw)


@pytest.mark.gpu
def test_calls_on_several_streams_at_once():
    """Calls that need the whole GPU at once, small ones and a linear layer, on four streams that do not wait for
    each other."""
    E, k = 64, 4
    logits = [_logits(T, E, 50 + T).to(DEV) for T in (40, 700, 6000, 20000)]
    x = torch.randn(300, 512, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    codes, scales = mx.mxfp4_quantize(torch.randn(640, 512, generator=torch.Generator().manual_seed(6)).to(DEV))
    want = [mx.moe_mxfp4_route_scored(l, k, n_groups=8, top_groups=4) for l in logits]
    y = mx.mxfp4_linear(x, codes, scales)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for r in range(6):
        for i, s in enumerate(streams):
            n = (i + r) % 4
            got.append((n, mx.moe_mxfp4_route_scored(logits[n], k, n_groups=8, top_groups=4, stream=s),
                        mx.mxfp4_linear(x, codes, scales, stream=s)))
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    for n, r, z in got:
        assert all(torch.equal(r[key], want[n][key]) for key in want[n])
        assert torch.equal(z, y)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [100, 700, 5000])
def test_nan_logits_do_not_count_for_their_group(score, T):
    """A few NaN among ordinary logits: a group's two largest values are those of its numbers."""
    E, G = 48, 4
    g = torch.Generator().manual_seed(T)
    l = torch.randn(T, E, generator=g) * 2
    l[torch.rand(T, E, generator=g) < 0.04] = float("nan")
    for bias in (None, _bias(E, 61)):
        for tg in (1, 2):
            _check(l, 5, score=score, bias=bias, n_groups=G, top_groups=tg, group_top=2)
            _check(l, 5, bf16=True, score=score, bias=bias, n_groups=G, top_groups=tg, group_top=2, renorm=False)
