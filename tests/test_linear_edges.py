"""The linear layer (mxfp4_linear) at the edges of its range."""
import numpy as np
import pytest
import torch

import oracle
import moe_expert_gemm_mxfp4_b200 as mx
from helpers import f64_of
from test_linear import ACTS, DEV, _weights, tolerance

# token counts that reach the few-token engine with one launch, with hi and lo in one MMA, with two MMAs, with several
# token tiles; and the many-token engine
TOKENS = [1, 5, 24, 100, 150, 600, 17000]


def _one_hot(N, K, at, code=0x2, scale=127):
    """MXFP4 weights of zeros but for `code` (0x2: 1.0) at (n, at[n]), every block scale `scale`."""
    codes = np.zeros((N, K // 2), dtype=np.uint8)
    for n, k in enumerate(at):
        if k is not None:
            codes[n, k // 2] = code << (4 * (k % 2))
    return torch.from_numpy(codes).to(DEV), torch.full((N, K // 32), scale, dtype=torch.uint8, device=DEV)


def _linear(x, codes, scales, act="none", **kw):
    y = mx.mxfp4_linear(x.to(DEV), codes, scales, act=ACTS[act], **kw)
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    return y.cpu()


# the patterns of bf16's largest values, 248 2^120 to 255 2^120
LARGEST = torch.arange(0x7F78, 0x7F80, dtype=torch.int16).view(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("M", TOKENS)
def test_largest_values_stay_finite(M):
    """One element at the top of bf16's range times a power of two: the result is the element's product, exactly
    (a sum of one nonzero term has no rounding), and finite where it fits bf16."""
    K, N = 96, 5
    vals = LARGEST[torch.arange(M) % 8] * torch.where(torch.arange(M) % 3 == 1, -1.0, 1.0).to(torch.bfloat16)
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    x[:, 41] = vals
    codes, scales = _one_hot(N, K, [41, None, 41, 7, 41])
    got = _linear(x, codes, scales)
    zero = torch.zeros(M, dtype=torch.bfloat16)
    assert torch.equal(got, torch.stack([vals, zero, vals, zero, vals], 1))
    # the same products from smaller factors: half of the element against a weight of 2, an eighth against 4 x 2
    for part, code, scale in ((0.5, 0x4, 127), (0.125, 0x6, 128)):
        x[:, 41] = (vals.float() * part).to(torch.bfloat16)
        codes, scales = _one_hot(N, K, [41, None, 41, 7, 41], code, scale)
        got = _linear(x, codes, scales)
        assert torch.equal(got, torch.stack([vals, zero, vals, zero, vals], 1))


@pytest.mark.gpu
@pytest.mark.parametrize("M", TOKENS)
def test_largest_values_through_the_gate(M):
    """gate 2 against the largest up, and the largest gate against up 0.5.  SiLU(2) is within 2^-16 of its value in
    fp32, the product and bf16 round once each: 2^-8 + 2^-15 of the result."""
    K, F = 64, 3
    big = LARGEST[torch.arange(M) % 8]
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    x[:, 3], x[:, 40] = 2.0, big
    # features: gate and up rows (3, 40); (40, 3) with half of x[3]'s weight; (None, 40)
    codes, scales = _one_hot(2 * F, K, [3, 40, None, 40, 3, 40])
    scales[F + 1] = 125                                              # up: 0.25 x 2
    got = _linear(x, codes, scales, "swiglu").double()
    b = big.double()
    want = torch.stack([2 / (1 + np.exp(-2.0)) * b, b * 0.5, torch.zeros(M, dtype=torch.float64)], 1)
    limit = torch.finfo(torch.bfloat16).max
    over = want > limit * (1 + 2.0 ** -9)                            # the first overflows: SiLU(2) is 1.76
    assert torch.isinf(got[over]).all()
    assert (torch.abs(got - want)[~over] <= (2.0 ** -8 + 2.0 ** -15) * want[~over]).all()
    x[:, 3] = 1.0                                                    # SiLU(1) = 0.73: all finite
    got = _linear(x, codes, scales, "swiglu").double()
    want = torch.stack([1 / (1 + np.exp(-1.0)) * b, b * 0.25, torch.zeros(M, dtype=torch.float64)], 1)
    assert (torch.abs(got - want) <= (2.0 ** -8 + 2.0 ** -15) * want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu", "swiglu"])
def test_tails_of_the_activations(M, act):
    """z from -110 to 110: the activations keep their relative accuracy down to bf16's smallest numbers.  The
    exponential's argument v carries at most 6 roundings (|v| <= 104 where the result is not 0: 104 * 6 * 2^-24, below
    2^-14 of the result), the hardware's exponential is off by (4 + 1.2 |v|) 2^-23, below 2^-15, the quotient and
    the products by less than 2^-20: 2^-13 together.  bf16 rounds once (2^-8, at the bottom half of 2^-133), and
    fp32 before the gate's product by 2^-150 at the bottom."""
    K = 96
    z = torch.linspace(-110, 110, 881).to(torch.bfloat16)
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    at = (88 + torch.arange(M)[:, None] * 97 + torch.arange(3) * 861) % 881   # the first row: z = -88, -93, -98
    x[:, [1, 34, 63]] = z[at]
    up = 1.0
    if act == "swiglu":   # the up rows read 2^40, in a block of its own
        x[:, 70] = up = 2.0 ** 40
        codes, scales = _one_hot(6, K, [1, 34, 63, 70, 70, 70])
    else:
        codes, scales = _one_hot(3, K, [1, 34, 63])
    got = _linear(x, codes, scales, act).double()
    v = z[at].double()
    if act == "gelu":
        want = 0.5 * v * torch.special.erfc(-v / 2 ** 0.5)
    elif act == "gelu_tanh":
        want = v * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    else:
        want = v * torch.sigmoid(v) * up
    tol = (2.0 ** -8 + 2.0 ** -13) * want.abs() + 2.0 ** -134 + 2.0 ** -150 * up
    bad = (got - want).abs() > tol
    assert not bad.any(), (v[bad][:5], got[bad][:5], want[bad][:5])
    if act == "swiglu":
        assert want.abs()[0, 0] > 1e-25              # far above the smallest numbers


@pytest.mark.gpu
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("act,N", [("none", 141), ("relu", 143), ("silu", 142), ("gelu", 141), ("gelu_tanh", 131),
                                   ("swiglu", 280), ("swiglu", 282), ("swiglu", 142)])
def test_infinities_and_nan_through_every_epilogue(M, act, N):
    """Inf and NaN in x, in block scales (gate and up rows), bias and residual come out where the formula has them, and
    nowhere else; beside them the results are the ordinary ones, within the bound of the parity tests."""
    K, inf, nan = 128, float("inf"), float("nan")
    n_out = N // 2 if act == "swiglu" else N
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    x[0, 3] = inf
    if M > 4:
        x[1, 70] = -inf
        x[2, 5], x[2, 9] = inf, -inf
        x[3, 64] = nan
    codes, scales = _weights(N, K, 4)
    scales = scales.copy()
    scales[7, 1] = scales[n_out - 1, 3] = scales[N - 1, 0] = scales[N - 12, 2] = 255
    bias = (torch.randn(N, generator=g) * 0.3).to(torch.bfloat16 if N % 2 else torch.float32)
    bias[2], bias[14], bias[N - 3], bias[N - 20], bias[n_out - 5] = inf, -inf, nan, inf, -inf
    res = torch.randn(M, n_out, generator=g).to(torch.bfloat16)
    res[0, 11], res[0, 12], res[M - 1, n_out - 7], res[M - 1, 20] = inf, nan, -inf, inf
    got = _linear(x, torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), act, bias=bias.to(DEV),
                  residual=res.to(DEV)).double().numpy()
    xf, b, r = f64_of(x), f64_of(bias), f64_of(res)
    W = oracle.dequantize_f64(codes, scales)
    assert np.isnan(W).any()
    with np.errstate(all="ignore"):
        z = torch.from_numpy(xf) @ torch.from_numpy(W).T + torch.from_numpy(b)
        if act == "swiglu":
            a = z[:, :n_out] / (1 + torch.exp(-z[:, :n_out])) * z[:, n_out:]
        else:
            a = dict(none=lambda v: v, relu=lambda v: torch.where(v < 0, 0.0, v), silu=lambda v: v / (1 + torch.exp(-v)),
                     gelu=lambda v: v * (1 + torch.erf(v / 2 ** 0.5)) / 2,
                     gelu_tanh=lambda v: v * (1 + torch.tanh((2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3))) / 2)[act](z)
        ref = a.numpy() + r
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    isinf = np.isinf(ref)
    assert isinf.any() and np.array_equal(got[isinf], ref[isinf])
    fin = np.isfinite(ref)
    assert np.isfinite(got[fin]).all()
    # the bound from finite stand-ins: an output is finite only where what is not finite did not reach it (or relu cut it off)
    xs, bs, rs = (np.where(np.isfinite(v), v, 0.0) for v in (xf, b, r))
    tol = tolerance(torch.from_numpy(xs), codes, np.where(scales == 255, 0, scales).astype(np.uint8), bs, act,
                    np.where(fin, ref, 0.0), rs)
    assert (np.abs(got[fin] - ref[fin]) <= tol[fin]).all()
