"""The linear layer with a fused epilogue (mxfp4_linear): the oracle against brute force and
the refusals (CPU); the outputs against the fp64 oracle within the rounding of the fp32
accumulation, of the activation and of the one rounding to bf16 (GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import moe_expert_gemm_mxfp4_b200 as mx
from moe_expert_gemm_mxfp4_b200 import _lib
from helpers import bits_of, f64_of

DEV = "cuda:0"
ACTS = dict(none=mx.ACT_NONE, relu=mx.ACT_RELU, silu=mx.ACT_SILU, gelu=mx.ACT_GELU, gelu_tanh=mx.ACT_GELU_TANH,
            swiglu=mx.ACT_SWIGLU)


# ---------------------------------------------------------------- oracle

@pytest.mark.parametrize("act", list(ACTS))
def test_oracle_against_fsum(act):
    g = np.random.default_rng(2)
    M, K, N = 3, 64, 6
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = g.integers(120, 130, (N, K // 32), dtype=np.uint8)
    bias, n_out = g.normal(size=N), N // 2 if act == "swiglu" else N
    res = g.normal(size=(M, n_out))
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6]

    def z(m, n):
        t = []
        for k in range(K):
            c = int(codes[n, k // 2]) >> (4 * (k % 2)) & 15
            t.append(float(x[m, k]) * (-1) ** (c >> 3) * grid[c & 7] * 2.0 ** (int(scales[n, k // 32]) - 127))
        return math.fsum(t) + bias[n]

    f = dict(none=lambda v: v, relu=lambda v: max(v, 0.0), silu=lambda v: v / (1 + math.exp(-v)),
             gelu=lambda v: v * (1 + math.erf(v / math.sqrt(2))) / 2,
             gelu_tanh=lambda v: v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))) / 2).get(act)
    got = oracle.linear(bits_of(x), codes, scales, bias, act, res)
    for m in range(M):
        for n in range(n_out):
            if act == "swiglu":
                want = z(m, n) / (1 + math.exp(-z(m, n))) * z(m, n + n_out)
            else:
                want = f(z(m, n))
            assert abs(got[m, n] - want - res[m, n]) <= 1e-10 * (1 + abs(want))


# ---------------------------------------------------------------- refusals (CPU)

A, U, N0 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001), ctypes.c_void_p(0)
FAR = ctypes.c_void_p(1 << 50)


def test_argument_checks():
    from moe_expert_gemm_mxfp4_b200 import build as mxbuild
    mxbuild.build()
    lib = _lib.load()

    def call(x=A, M=8, K=256, c=A, s=A, N=512, bias=N0, bdt=0, act=0, res=N0, y=FAR, ws=A, nbytes=1 << 40):
        return lib.mxfp4_linear(x, M, K, c, s, N, bias, bdt, act, res, y, ws, nbytes, N0)

    for kw in (dict(x=N0), dict(c=N0), dict(s=N0), dict(y=N0), dict(M=0), dict(K=0), dict(N=0), dict(M=-1), dict(N=-5),
               dict(act=6), dict(act=-1), dict(bias=A, bdt=2)):
        assert call(**kw) == _lib.ERR_INVALID_ARG, kw
    for kw in (dict(K=48), dict(K=(1 << 20) + 32), dict(M=1 << 31), dict(N=1 << 31), dict(N=511, act=5),
               dict(M=(1 << 31) - 1, N=(1 << 31) - 2)):
        assert call(**kw) == _lib.ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=U), dict(c=U), dict(s=U), dict(y=U), dict(bias=U), dict(res=U), dict(ws=U)):
        assert call(**kw) == _lib.ERR_MISALIGNED, kw
    for M in (1, 64, 8192):
        need = mx.mxfp4_linear_workspace_size(M, 2880, 5760, mx.ACT_SWIGLU)
        if need:
            assert call(M=M, K=2880, N=5760, act=5, nbytes=need - 1) == _lib.ERR_WORKSPACE
            assert call(M=M, K=2880, N=5760, act=5, ws=N0, nbytes=0) == _lib.ERR_WORKSPACE
    assert mx.mxfp4_linear_workspace_size(0, 2880, 5760) == 0
    # y over x, or over a residual that is not y itself: 64 x 256 of x, 64 x 512 of y and residual.  What passes
    # this check is refused by the next, for a workspace of nothing: no call here may launch on made-up addresses.
    at = ctypes.c_void_p
    base, far, x_bytes, y_bytes = 1 << 30, 1 << 40, 64 * 256 * 2, 64 * 512 * 2
    assert mx.mxfp4_linear_workspace_size(64, 256, 512) > 0

    def placed(**kw):
        return call(M=64, nbytes=0, **kw)

    for y in (base, base + 16, base + x_bytes - 16, base - y_bytes + 16):
        assert placed(x=at(base), y=at(y)) == _lib.ERR_INVALID_ARG
    for y in (base + 16, base + y_bytes - 16, base - y_bytes + 16):
        assert placed(x=at(far), res=at(base), y=at(y)) == _lib.ERR_INVALID_ARG
    for y in (base + x_bytes, base - y_bytes):
        assert placed(x=at(base), y=at(y)) == _lib.ERR_WORKSPACE
    for y in (base, base + y_bytes, base - y_bytes):
        assert placed(x=at(far), res=at(base), y=at(y)) == _lib.ERR_WORKSPACE


def test_binding_refusals():
    u8, bf16 = torch.uint8, torch.bfloat16
    x, c, s = torch.zeros(4, 64, dtype=bf16), torch.zeros(6, 32, dtype=u8), torch.zeros(6, 2, dtype=u8)
    f = mx.mxfp4_linear
    with pytest.raises(ValueError, match="x: expected dtype"):
        f(x.float(), c, s)
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(64, 4, dtype=bf16).t(), c, s)
    with pytest.raises(ValueError, match="w_codes: expected shape"):
        f(x, torch.zeros(6, 31, dtype=u8), s)
    with pytest.raises(ValueError, match="w_scales: expected shape"):
        f(x, c, torch.zeros(6, 1, dtype=u8))
    with pytest.raises(ValueError, match="bias: expected shape"):
        f(x, c, s, bias=torch.zeros(5))
    with pytest.raises(ValueError, match="bias: expected dtype"):
        f(x, c, s, bias=torch.zeros(6, dtype=torch.float64))
    with pytest.raises(ValueError, match="residual: expected shape"):
        f(x, c, s, act=mx.ACT_SWIGLU, residual=torch.zeros(4, 6, dtype=bf16))
    with pytest.raises(ValueError, match="residual: expected dtype"):
        f(x, c, s, residual=torch.zeros(4, 6))
    with pytest.raises(ValueError, match="out: expected shape"):
        f(x, c, s, out=torch.zeros(4, 5, dtype=bf16))
    with pytest.raises(ValueError, match="even number"):
        f(x, torch.zeros(5, 32, dtype=u8), torch.zeros(5, 2, dtype=u8), act=mx.ACT_SWIGLU)
    with pytest.raises(ValueError, match="CUDA"):
        f(x, c, s)


# ---------------------------------------------------------------- parity (GPU)

def _weights(N, K, seed, w_std=0.02):
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(seed)) * w_std
    return oracle.quantize(w.numpy(), oracle.FLOOR)


def tolerance(x, codes, scales, bias, act, ref, res):
    """Elementwise bound of |y - ref|.  With a = sum |x w| + |bias|: the fp32 accumulation in any
    order is off by at most K 2^-24 a (as the router projection's logits); operands that are kept
    in parts may leave out 2^-21 of the largest |x| of a 32-block times the block's |w|; the
    activation (slope at most 1.13) passes that on and adds 2^-20 of itself, the gated one by
    the product rule; the sum with the residual rounds twice (fp32 2^-24, bf16 2^-8)."""
    xf, W = np.abs(f64_of(x)), np.abs(oracle.dequantize_f64(codes, scales))
    M, K = xf.shape
    a = xf @ W.T + (0 if bias is None else np.abs(bias))
    amax = xf.reshape(M, K // 32, 32).max(-1)
    e = K * 2.0 ** -24 * a + 2.0 ** -21 * amax @ W.reshape(-1, K // 32, 32).sum(-1).T
    if act == "swiglu":
        h = a.shape[1] // 2
        e = 1.13 * e[:, :h] * (a[:, h:] + e[:, h:]) + a[:, :h] * e[:, h:] + 2.0 ** -20 * a[:, :h] * a[:, h:]
    else:
        e = 1.13 * e + 2.0 ** -20 * a
    r = 0 if res is None else np.abs(res)
    return 2.0 ** -8 * (np.abs(ref) + e) + e + 2.0 ** -23 * (np.abs(ref) + r) + 2.0 ** -133


def _check(x, codes, scales, act="none", bias=None, res=None, **kw):
    c, s = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    y = mx.mxfp4_linear(x.to(DEV), c, s, bias=None if bias is None else bias.to(DEV), act=ACTS[act],
                        residual=None if res is None else res.to(DEV), **kw)
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    b, r = (None if t is None else f64_of(t) for t in (bias, res))
    ref = oracle.linear(bits_of(x), codes, scales, b, act, r)
    got = f64_of(y)
    assert got.shape == ref.shape and np.isfinite(got).all()
    tol = tolerance(x, codes, scales, b, act, ref, r)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])
    # the bound counts worst cases; what random operands give is far smaller: most of the error is the last rounding
    if np.abs(ref).max() > 0:
        assert np.linalg.norm(got - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    return y


def _case(M, K, N, act, bias, residual, seed=0, std=1.0):
    g = torch.Generator().manual_seed(M * 31 + K * 7 + N + seed)
    x = (torch.randn(M, K, generator=g) * std).to(torch.bfloat16)
    codes, scales = _weights(N, K, seed + N)
    b = None if bias is None else (torch.randn(N, generator=g) * 0.3).to(bias)
    n_out = N // 2 if act == "swiglu" else N
    r = torch.randn(M, n_out, generator=g).to(torch.bfloat16) if residual else None
    return x, codes, scales, act, b, r


# one token to more than the largest token tile, K of one block to several stages with every
# remainder of a stage, N of one row and off every multiple of a tile and of a vector
SHAPES = [(1, 32, 1), (1, 64, 2), (2, 32, 130), (3, 96, 64), (7, 160, 258), (8, 256, 128), (9, 2880, 66), (16, 352, 200),
          (17, 128, 384), (31, 512, 100), (32, 1056, 130), (33, 64, 1000), (64, 2880, 512), (65, 224, 126), (77, 1056, 1002),
          (128, 416, 254), (129, 320, 258), (200, 1024, 640), (256, 288, 514), (257, 96, 130), (300, 2880, 290),
          (512, 544, 600), (513, 192, 256), (600, 2080, 1026), (1030, 704, 770)]


# many tokens with little K (the tile's epilogue is all there is), one output column, columns past the
# last full tile of every width, and few tokens with more K than the few-token engine takes
SHAPES += [(1100, 32, 1), (900, 64, 40), (2049, 96, 130), (600, 160, 1950), (1025, 32, 2880), (1537, 128, 514),
           (777, 256, 1300), (3, 8224, 70), (40, 9216, 131)]
# two rounds of the few-token engine, ten token tiles of it; the other engine with little to do per tile
SHAPES += [(300, 2048, 9500), (1100, 672, 1536), (16700, 32, 40), (20000, 64, 1), (2600, 160, 1950), (5000, 64, 514),
           (2049, 96, 1300), (6000, 96, 258), (4000, 128, 515), (1400, 256, 1550), (9000, 32, 130)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_against_oracle(M, K, N):
    _check(*_case(M, K, N, "none", None, False))
    _check(*_case(M, K, N, "none", torch.bfloat16, True, seed=1))
    if N % 2 == 0:
        _check(*_case(M, K, N, "swiglu", torch.bfloat16, False, seed=2))
        _check(*_case(M, K, N, "swiglu", None, True, seed=3))


@pytest.mark.gpu
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,K,N", [(5, 96, 70), (70, 160, 300), (700, 256, 302), (6000, 96, 302)])
def test_activations(act, M, K, N):
    for bias in (torch.float32, torch.bfloat16):
        _check(*_case(M, K, N, act, bias, bias == torch.float32, seed=5, std=4.0))


# every route through the sizes, at odd N (rows that no vector is aligned to)
@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 100, 400, 1500, 2700])
def test_odd_rows(M):
    _check(*_case(M, 288, 1001, "gelu_tanh", torch.float32, True))
    _check(*_case(M, 288, 1002, "swiglu", torch.float32, True))   # n_out = 501


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 150, 600, 1100, 17000])
def test_wide_range_of_scales(M):
    """Block scales and activations over many powers of two, zero blocks among them."""
    K, N = 320, 200
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-12, 12, (M, K // 32), generator=g).float()).repeat_interleave(32, 1)
    x[:, 32:64] = 0
    r = np.random.default_rng(M)
    codes = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = r.integers(107, 147, (N, K // 32), dtype=np.uint8)
    scales[::7] = 0                    # 2^-127
    _check(x.to(torch.bfloat16), codes, scales)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 150, 600, 1100, 17000])
def test_outliers_inside_a_block(M):
    """One element of a block 2^12 times the others: the small ones still count in full."""
    K, N = 256, 130
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g)
    x[:, 5::32] *= 4096
    codes, scales = _weights(N, K, 9)
    _check(x.to(torch.bfloat16), codes, scales)
    codes[:, 2::16] &= 0x0F            # the outlier meets a weight of 0
    _check(x.to(torch.bfloat16), codes, scales)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 150, 600, 1100, 17000])
def test_exact_products(M):
    """Powers of two and small whole numbers add without rounding: the result is the formula's."""
    K, N = 192, 96
    g = torch.Generator().manual_seed(M + 1)
    x = torch.randint(-8, 9, (M, K), generator=g).to(torch.bfloat16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).numpy()
    scales = np.full((N, K // 32), 127, dtype=np.uint8)
    y = mx.mxfp4_linear(x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    ref = oracle.linear(bits_of(x), codes, scales)
    assert np.array_equal(bits_of(y), oracle.f64_to_bf16(ref))
    # every bf16 pattern of a significand, one element per token against a weight of 1
    x = torch.zeros(max(M, 1), 64, dtype=torch.bfloat16)
    vals = (torch.arange(M * 2) % 256 + 128).to(torch.float32) * torch.exp2((torch.arange(M * 2) % 37 - 20).float())
    x[:, 3], x[:, 40] = vals[:M].to(torch.bfloat16), vals[M:].to(torch.bfloat16)
    codes = np.zeros((2, 32), dtype=np.uint8)
    codes[0, 1], codes[1, 20] = 0x20, 0x02
    y = mx.mxfp4_linear(x.to(DEV), torch.from_numpy(codes).to(DEV), torch.full((2, 2), 127, dtype=torch.uint8, device=DEV))
    assert torch.equal(y.cpu(), torch.stack([x[:, 3], x[:, 40]], 1))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24, 150, 600, 1100, 17000])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_infinities_and_nan(M, act):
    K, N = 128, 140
    g = torch.Generator().manual_seed(M + 2)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    inf, nan = float("inf"), float("nan")
    x[0, 3] = inf
    if M > 4:
        x[1, 70] = -inf
        x[2, 5], x[2, 9] = inf, -inf
        x[3, 64] = nan
        x[4] = 3e38
    codes, scales = _weights(N, K, 4)
    scales = scales.copy()
    scales[7, 1] = 255                 # a weight block of NaN
    res = torch.randn(M, N, generator=g).to(torch.bfloat16)
    res[0, 11], res[0, 12] = inf, nan
    y = mx.mxfp4_linear(x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), act=ACTS[act],
                        residual=res.to(DEV))
    torch.cuda.synchronize()
    # the plain form, in fp32 (where 3e38 overflows as in the kernel's sums, whatever their order: the test
    # compares that row's finite values with nothing)
    W = torch.from_numpy(oracle.dequantize_f64(codes, scales)).float()
    z = x.float() @ W.t()
    z = torch.where(z < 0, 0.0, z) if act == "relu" else z
    ref = (z + res.float()).to(torch.bfloat16)
    got = y.cpu()
    rows = [r for r in range(M) if r != 4]
    assert torch.equal(torch.isnan(got[rows]), torch.isnan(ref[rows]))
    isinf = torch.isinf(ref[rows])
    assert torch.equal(got[rows][isinf], ref[rows][isinf])
    fin = torch.isfinite(ref[rows])
    assert torch.isfinite(got[rows][fin]).all()
    assert torch.allclose(got[rows][fin].float(), ref[rows][fin].float(), rtol=2 ** -7, atol=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 64, 300, 1200, 6000])
def test_residual_in_place(M):
    x, codes, scales, act, b, r = _case(M, 320, 260, "silu", torch.bfloat16, True)
    want = _check(x, codes, scales, act, b, r)
    buf = r.to(DEV)
    args = (x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    out = mx.mxfp4_linear(*args, bias=b.to(DEV), act=ACTS[act], residual=buf, out=buf)
    assert out is buf and torch.equal(buf, want)


@pytest.mark.gpu
def test_output_over_the_input_is_refused():
    x, codes, scales, _, _, r = _case(5, 128, 128, "none", None, True)
    c, s = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    both = torch.cat([x, r]).to(DEV)
    for kw in (dict(out=both[:5]), dict(out=both[1:6]), dict(out=both[4:9], residual=both[5:])):
        with pytest.raises(mx.Mxfp4Error):
            mx.mxfp4_linear(both[:5] if "residual" not in kw else x.to(DEV), c, s, **kw)
    y = mx.mxfp4_linear(both[:5], c, s, residual=both[5:], out=both[5:])   # the rows behind x, in place
    assert torch.equal(y, mx.mxfp4_linear(x.to(DEV), c, s, residual=r.to(DEV)))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,act", [(1, 64, 3, "none"), (19, 352, 201, "none"), (77, 160, 130, "swiglu"),
                                       (300, 288, 257, "none"), (1025, 96, 258, "swiglu"), (1100, 544, 1003, "none"),
                                       (17000, 96, 130, "swiglu"), (6000, 96, 258, "none"), (4000, 128, 515, "none")])
def test_stays_inside_output_and_workspace(M, K, N, act):
    from test_guard_gpu import Guarded
    x, codes, scales, act, b, r = _case(M, K, N, act, torch.float32, True)
    n_out = N // 2 if act == "swiglu" else N
    need = mx.mxfp4_linear_workspace_size(M, K, N, ACTS[act])
    out, ws = Guarded((M, n_out), torch.bfloat16), Guarded((max(need, 16),), torch.uint8)
    _check(x, codes, scales, act, b, r, out=out.t, ws=ws.t)
    out.check("y")
    ws.check("workspace")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 96, 700, 1300, 5700])
def test_own_stream_and_graph(M):
    x, codes, scales, act, b, r = _case(M, 480, 330, "swiglu", torch.bfloat16, True)
    c, s, b, r = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), b.to(DEV), r.to(DEV)
    buf = x.to(DEV)
    want = mx.mxfp4_linear(buf, c, s, bias=b, act=ACTS[act], residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mxfp4_linear(buf, c, s, bias=b, act=ACTS[act], residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = mx.mxfp4_linear(buf, c, s, bias=b, act=ACTS[act], residual=r)
    buf.copy_(torch.randn(M, 480))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, mx.mxfp4_linear(buf, c, s, bias=b, act=ACTS[act], residual=r))


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    """Calls of both engines that overlap on the GPU, each with its own workspace."""
    cases = [_case(M, 320, 520, "swiglu", torch.bfloat16, True, seed=M) for M in (4, 70, 640, 3600)]
    dev = []
    for x, codes, scales, act, b, r in cases:
        dev.append((x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), b.to(DEV), r.to(DEV)))

    def call(i, stream=None):
        x, c, s, b, r = dev[i]
        return mx.mxfp4_linear(x, c, s, bias=b, act=mx.ACT_SWIGLU, residual=r, stream=stream)

    want = [call(i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [[call((i + k) % 4, streams[i]) for i in range(4)] for k in range(8)]
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    for k in range(8):
        for i in range(4):
            assert torch.equal(got[k][i], want[(i + k) % 4])


def test_both_engines_are_in_the_shapes():
    """The workspace tells which engine a size goes to: the one for many tokens holds the weights in bf16."""
    from moe_expert_gemm_mxfp4_b200 import build as mxbuild
    mxbuild.build()

    def many(M, K, N, act="none"):
        return mx.mxfp4_linear_workspace_size(M, K, N, ACTS[act]) == (N * K * 2 + 255) // 256 * 256

    assert 8 <= sum(many(*s) for s in SHAPES) <= len(SHAPES) - 20
    assert many(6000, 96, 302) and many(17000, 320, 200) and many(17000, 256, 130) and many(17000, 192, 96)
    assert many(17000, 128, 140) and many(2700, 288, 1001) and many(2700, 288, 1002, "swiglu") and many(6000, 320, 260)
    assert many(17000, 96, 130, "swiglu") and many(4000, 128, 515) and many(5700, 480, 330, "swiglu")
    assert many(3600, 320, 520, "swiglu") and not many(300, 2048, 9500) and not many(1100, 672, 1536)


def test_workspace_sizes():
    """Nothing up to 16 tokens of a short contraction; then the prepared activations and scales, which
    grow with the tokens; then the weights in bf16, whatever the tokens."""
    from moe_expert_gemm_mxfp4_b200 import build as mxbuild
    mxbuild.build()
    size = mx.mxfp4_linear_workspace_size
    assert size(1, 2880, 2880) == size(16, 2880, 2880) == 0
    few = [size(M, 2880, 2880) for M in (17, 64, 112, 256, 384)]
    assert all(a < b for a, b in zip(few, few[1:])) and few[-1] < 2 * 2880 * 2880
    assert size(1024, 2880, 2880) == size(8192, 2880, 2880) == 2 * 2880 * 2880
    assert size(8192, 2880, 5760, mx.ACT_SWIGLU) == 2 * 2880 * 5760
    assert size(2, 8224, 64) == 2 * 8224 * 64
