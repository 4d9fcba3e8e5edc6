"""The scored routing and the linear layer together with the layer's parts, as a model with a scored
router and a shared expert runs them:
    r = route_scored(logits);  routed = combine(experts(gather(x)));
    out = down(SwiGLU(up(x))) + routed
against the fp64 oracle; the same chain captured and replayed; and the expert-parallel layer with a
scored router."""
import datetime
import os
import socket

import numpy as np
import pytest
import torch

import oracle
import moe_expert_gemm_mxfp4_b200 as mx
from moe_expert_gemm_mxfp4_b200 import ep, inputs
from helpers import assert_close_tol, bits_of, f64_of

DEV = "cuda:0"
ROUTER = dict(score=mx.SCORE_SIGMOID, n_groups=4, top_groups=2, group_top=2, renorm=True, scale=2.5)


def _layer(T, H, I, E, seed):
    cfg = inputs.MoEConfig("scored", seed=seed, T=T, E=E, H=H, I=I, w_std=0.05)
    x, logits = inputs.moe_activations(cfg)
    q13 = [oracle.quantize(inputs.expert_weights(cfg, e)[0].numpy()) for e in range(E)]
    q2 = [oracle.quantize(inputs.expert_weights(cfg, e)[1].numpy()) for e in range(E)]
    w = [np.stack([a for a, _ in q13]), np.stack([b for _, b in q13]), np.stack([a for a, _ in q2]),
         np.stack([b for _, b in q2])]
    up = oracle.quantize(inputs.seeded_f32((2 * I, H), seed + 1, 0.05).numpy())
    down = oracle.quantize(inputs.seeded_f32((H, I), seed + 2, 0.05).numpy())
    bias = inputs.seeded_f32((E,), seed + 3, 0.05)
    up_bias = inputs.seeded_bf16((2 * I,), seed + 4, 0.1)
    return x, logits, w, up, down, bias, up_bias


def _dev(a):
    return (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(DEV)


def _run(x, logits, w, up, down, bias, up_bias, k):
    r = mx.moe_mxfp4_route_scored(logits, k, bias=bias, **ROUTER)
    xs = mx.mxfp4_gather_rows(x, r["perm"], k)
    ws = mx.mxfp4_gather_rows(r["weights"].reshape(-1, 1), r["perm"], 1).reshape(-1)
    routed = mx.moe_mxfp4_combine(mx.moe_mxfp4_experts(xs, r["offsets"], ws, *w), r["inv"], k)
    h = mx.mxfp4_linear(x, *up, bias=up_bias, act=mx.ACT_SWIGLU)
    return r, mx.mxfp4_linear(h, *down, residual=routed)


def _oracle(x, logits, w, up, down, bias, up_bias, k):
    r = oracle.route_scored(logits.double().numpy(), k, "sigmoid", bias.double().numpy(), 4, 2, 2, True, 2.5)
    xf = f64_of(x)
    routed = np.zeros_like(xf)
    I = w[2].shape[2] * 2
    for e in np.unique(r["ids"]):
        rows, slots = np.nonzero(r["ids"] == e)
        W13, W2 = oracle.dequantize_f64(w[0][e], w[1][e]), oracle.dequantize_f64(w[2][e], w[3][e])
        g = xf[rows] @ W13.T
        h = oracle.bf16_to_f64(oracle.f64_to_bf16(oracle.silu(g[:, :I]) * g[:, I:]))
        np.add.at(routed, rows, r["w"][rows, slots][:, None] * (h @ W2.T))
    routed = oracle.bf16_to_f64(oracle.f64_to_bf16(routed))
    h = oracle.f64_to_bf16(oracle.linear(bits_of(x), *up, f64_of(up_bias), "swiglu"))
    return r, oracle.linear(h, *down, residual=routed)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 8, 2), (37, 192, 128, 16, 4), (300, 256, 320, 32, 6), (1300, 128, 192, 8, 3)])
def test_layer_with_scored_router_and_shared_expert(T, H, I, E, k):
    host = _layer(T, H, I, E, seed=T + I)
    dev = [tuple(map(_dev, a)) if isinstance(a, (tuple, list)) else _dev(a) for a in host]
    r, out = _run(*dev, k)
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    ref, want = _oracle(*host, k)
    for key in ("ids", "counts", "offsets", "perm", "inv"):
        assert np.array_equal(r[key].cpu().numpy(), ref[key])
    # the layer's bar: three products with bf16 roundings between them
    assert_close_tol(f64_of(out), want, what=f"layer T={T}")
    # captured and replayed on other inputs
    x, logits = dev[0].clone(), dev[1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, cap = _run(x, logits, *dev[2:], k)
    x.copy_(torch.flip(dev[0], [0]))
    logits.copy_(torch.flip(dev[1], [0]))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, _run(x, logits, *dev[2:], k)[1])


def test_expert_parallel_ops_take_a_router(monkeypatch):
    seen = {}

    def scored(logits, top_k, **kw):
        seen.update(kw, top_k=top_k)
        return "scored"

    monkeypatch.setattr(mx, "moe_mxfp4_route_scored", scored)
    monkeypatch.setattr(mx, "moe_mxfp4_route", lambda logits, top_k: "plain")
    assert ep.LibraryOps().route(None, 4) == "plain"
    assert ep.LibraryOps(router=ROUTER).route(None, 6) == "scored"
    assert seen == dict(ROUTER, top_k=6)


@pytest.mark.gpu
def test_expert_parallel_layer_with_a_scored_router():
    import torch.distributed as dist
    T, H, I, E, k = 96, 256, 192, 8, 2
    x, logits, w, _, _, bias, _ = _layer(T, H, I, E, seed=5)
    x, logits, w, router = x.to(DEV), logits.to(DEV), list(map(_dev, w)), dict(ROUTER, bias=bias.to(DEV))
    r = mx.moe_mxfp4_route_scored(logits, k, **router)
    ws = mx.mxfp4_gather_rows(r["weights"].reshape(-1, 1), r["perm"], 1).reshape(-1)
    want = mx.moe_mxfp4_combine(mx.moe_mxfp4_experts(mx.mxfp4_gather_rows(x, r["perm"], k), r["offsets"], ws, *w), r["inv"], k)
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    os.environ["MASTER_ADDR"], os.environ["MASTER_PORT"] = "127.0.0.1", str(port)
    os.environ.setdefault("NCCL_NVLS_ENABLE", "0")
    dist.init_process_group("nccl", rank=0, world_size=1, timeout=datetime.timedelta(seconds=60),
                            device_id=torch.device(DEV))
    try:
        out = ep.moe_mlp_ep(x, logits, k, w, ep.ExpertPartition(E, 1), 0, ops=ep.LibraryOps(router=router))
        torch.cuda.synchronize()
    finally:
        dist.destroy_process_group()
    assert np.array_equal(bits_of(out), bits_of(want))
