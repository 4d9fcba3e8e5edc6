"""Cases that measure the routing with scores (moe_mxfp4_route_scored) and the MXFP4 linear
layer with a fused epilogue (mxfp4_linear): what a mixture-of-experts model with a scored
router and a shared expert runs around its expert GEMMs.

``run`` computes the plain form, in elementary torch operations, unless ``own`` is set, when
it makes the library's calls."""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _route(name, T, E, k, dtype="f32", score="softmax", bias=False, groups=1, top_groups=1, group_top=1,
           renorm=True, scale=1.0, masked=False):
    return dict(name=name, op="route", T=T, E=E, k=k, dtype=dtype, score=score, bias=bias, groups=groups,
                top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale, masked=masked)


def _linear(name, M, K, N, act="none", bias="none", residual=False):
    return dict(name=name, op="linear", M=M, K=K, N=N, act=act, bias=bias, residual=residual)


def listed():
    return [
        # one token of a 32-expert layer: nothing but latency
        _route("route token", 1, 32, 4),
        # a decode batch through a sigmoid router with a balance bias, 4 of 8 groups kept
        _route("route decode", 64, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2,
               scale=2.5),
        # a ragged prompt, bf16 logits, a group count that is no power of two, some experts switched off
        _route("route odd", 1237, 90, 6, dtype="bf16", bias=True, groups=6, top_groups=3, renorm=False,
               masked=True),
        # a prefill chunk through the same sigmoid router
        _route("route prefill", 8192, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2,
               scale=2.5),
        # the largest batch: softmax over 128 experts, no bias
        _route("route long", 65536, 128, 4, dtype="bf16"),
        # one token: the down projection of a shared expert, added to the routed experts' output
        _linear("linear token", 1, 2880, 2880, residual=True),
        # a decode batch: the gated up projection of a shared expert with biases
        _linear("linear decode", 64, 2880, 5760, act="swiglu", bias="bf16"),
        # ragged everything: 32-element tail in K, odd N, fp32 bias, tanh GELU and residual
        _linear("linear odd", 77, 1056, 1001, act="gelu_tanh", bias="f32", residual=True),
        # a short prompt through a plain projection
        _linear("linear short", 512, 2880, 2880, act="silu", bias="bf16"),
        # a long contraction: the down projection of a wide dense layer
        _linear("linear wide", 2048, 7680, 2880, residual=True),
        # prefill: the gated up projection of a shared expert, the largest call
        _linear("linear prefill", 8192, 2880, 5760, act="swiglu", bias="bf16"),
        # prefill: its down projection
        _linear("linear down", 8192, 2880, 2880, bias="bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        E = _log(rng, 8, 256)
        groups = rng.choice([g for g in range(1, 33) if E % g == 0 and (g == 1 or E // g >= 2)])
        top_groups = rng.randint(1, groups)
        c = _route("", _log(rng, 1, 65536), E, rng.randint(1, min(8, top_groups * (E // groups))),
                   dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                   bias=rng.random() < 0.6, groups=groups, top_groups=top_groups,
                   group_top=rng.choice([1, 2]) if groups > 1 else 1, renorm=rng.random() < 0.7,
                   scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.3)
    else:
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu"])
        M, K, N = _log(rng, 1, 8192), 32 * _log(rng, 2, 240), _log(rng, 8, 11520)
        N += N % 2 if act == "swiglu" else 0
        most = 8192 * 2880 * 5760
        M = max(1, min(M, most // (K * N)))
        c = _linear("", M, K, N, act=act, bias=rng.choice(["none", "bf16", "f32"]), residual=rng.random() < 0.5)
    del c["name"]
    return c


def _quantized_weights(N, K, gen):
    """Normal weights as MXFP4: E2M1 codes of 32-element blocks, two to a byte (the even element
    in the low nibble), and one power-of-two scale byte per block."""
    w = torch.randn(N, K // 32, 32, device="cuda", generator=gen) * 0.02
    s = torch.floor(torch.log2(w.abs().amax(-1, keepdim=True))) - 2
    r = w * torch.exp2(-s)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(r.abs(), edges).to(torch.uint8) | ((r < 0).to(torch.uint8) << 3)
    code = code.reshape(N, K // 2, 2)
    codes = code[..., 0] | (code[..., 1] << 4)
    return codes.contiguous(), (s.reshape(N, K // 32) + 127).to(torch.uint8).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = randn(T, E) * 1.5 + 0.3 * randn(1, E)      # some experts are liked better by every token
        if case["masked"]:
            logits[:, E - max(1, E // 16):] = float("-inf")  # experts that are switched off
        st["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        # a balance bias moves the choice by a few per cent of a score
        st["bias_t"] = None
        if case["bias"]:
            st["bias_t"] = randn(E) * (0.05 if case["score"] == "sigmoid" else 0.3 / E)
        return st
    M, K, N = case["M"], case["K"], case["N"]
    st["x"] = randn(M, K).to(torch.bfloat16)
    st["codes"], st["scales"] = _quantized_weights(N, K, gen)
    st["bias_t"] = None
    if case["bias"] != "none":
        st["bias_t"] = (randn(N) * 0.1).to(torch.bfloat16 if case["bias"] == "bf16" else torch.float32)
    st["res_t"] = None
    if case["residual"]:
        st["res_t"] = randn(M, N // 2 if case["act"] == "swiglu" else N).to(torch.bfloat16)
    return st


def run(state):
    if own:
        import moe_expert_gemm_mxfp4_b200 as mx
        if state["op"] == "route":
            return mx.moe_mxfp4_route_scored(
                state["logits"], state["k"],
                score=mx.SCORE_SIGMOID if state["score"] == "sigmoid" else mx.SCORE_SOFTMAX, bias=state["bias_t"],
                n_groups=state["groups"], top_groups=state["top_groups"], group_top=state["group_top"],
                renorm=state["renorm"], scale=state["scale"])
        act = dict(none=mx.ACT_NONE, relu=mx.ACT_RELU, silu=mx.ACT_SILU, gelu=mx.ACT_GELU,
                   gelu_tanh=mx.ACT_GELU_TANH, swiglu=mx.ACT_SWIGLU)[state["act"]]
        return mx.mxfp4_linear(state["x"], state["codes"], state["scales"], bias=state["bias_t"], act=act,
                               residual=state["res_t"])
    return _plain_route(state) if state["op"] == "route" else _plain_linear(state)


def _plain_route(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    ninf = float("-inf")
    lg = st["logits"].double()        # the choice goes by 64 bits: scores next to each other must not swap
    off = lg == ninf
    if st["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-lg))
    else:
        m = lg.amax(-1, keepdim=True)
        e = torch.exp(lg - torch.where(m == ninf, 0.0, m))
        s = e / e.sum(-1, keepdim=True)
    s = torch.where(off, 0.0, s)
    c = s if st["bias_t"] is None else s + st["bias_t"].double()
    c = torch.where(off, ninf, c)
    if G > 1:
        top = c.view(T, G, E // G).sort(-1, descending=True).values
        v = top[..., 0]
        if st["group_top"] == 2:
            v = v + torch.where(top[..., 1] == ninf, 0.0, top[..., 1])
        kept = v.sort(dim=-1, descending=True, stable=True).indices[:, :st["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        keep = keep.repeat_interleave(E // G, 1)
        # experts that are off but in a kept group come before those of the other groups
        rank = torch.where(keep, torch.where(c == ninf, -1e300, c), -2e300)
        ids = rank.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    else:
        ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if st["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / torch.where(total == 0, 1.0, total))
    w = w * st["scale"]
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    perm = flat.sort(stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=perm.device)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    i32 = torch.int32
    return dict(ids=ids.to(i32), weights=w.float(), counts=counts.to(i32), offsets=offsets.to(i32),
                perm=perm.to(i32), inv=inv.to(i32))


def _plain_linear(st):
    table = torch.tensor([*E2M1, *(-v for v in E2M1)], device="cuda")
    codes, scales = st["codes"], st["scales"]
    N, K = codes.shape[0], 2 * codes.shape[1]
    pairs = torch.stack([codes & 15, codes >> 4], -1).int()
    w = table[pairs.view(N, K // 32, 32)] * torch.exp2(scales.float() - 127).unsqueeze(-1)
    z = st["x"].float() @ w.view(N, K).t()
    if st["bias_t"] is not None:
        z = z + st["bias_t"].float()
    act = st["act"]
    if act == "relu":
        z = z.clamp_min(0)
    elif act == "silu":
        z = z / (1 + torch.exp(-z))
    elif act == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    elif act == "gelu_tanh":
        z = 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    elif act == "swiglu":
        g, u = z[:, :N // 2], z[:, N // 2:]
        z = g / (1 + torch.exp(-g)) * u
    if st["res_t"] is not None:
        z = z + st["res_t"].float()
    return z.to(torch.bfloat16)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        item = 2 if case["dtype"] == "bf16" else 4
        # logits and bias read; ids, weights, perm, inv, counts and offsets written
        return {"bytes": T * E * item + (4 * E if case["bias"] else 0) + 16 * T * k + 4 * (2 * E + 1),
                "flops": 4 * T * E}
    M, K, N = case["M"], case["K"], case["N"]
    No = N // 2 if case["act"] == "swiglu" else N
    size = {"none": 0, "bf16": 2, "f32": 4}[case["bias"]]
    return {"bytes": 2 * M * K + N * K // 2 + N * K // 32 + size * N + 2 * M * No * (2 if case["residual"] else 1),
            "flops": 2 * M * N * K}


def exact(case, seed):
    """The definitions in 64 bits, written apart from the plain forms."""
    st = prepare(case, seed)
    if case["op"] == "route":
        w = torch.cat([_exact_weights(case, part, st["bias_t"]) for part in st["logits"].split(4096)])
        return dict(ids=None, weights=w, counts=None, offsets=None, perm=None, inv=None)
    W = _exact_dequantize(st["codes"], st["scales"])
    bias = torch.zeros(case["N"], dtype=torch.float64, device="cuda") if st["bias_t"] is None else st["bias_t"].double()
    z = torch.addmm(bias, st["x"].double(), W.T)
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    if case["act"] == "swiglu":
        z = silu(z[:, :case["N"] // 2]) * z[:, case["N"] // 2:]
    elif case["act"] == "silu":
        z = silu(z)
    elif case["act"] == "relu":
        z = torch.maximum(z, torch.zeros_like(z))
    elif case["act"] == "gelu":
        z = z * 0.5 * torch.erfc(-z / math.sqrt(2))
    elif case["act"] == "gelu_tanh":
        z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z if st["res_t"] is None else z + st["res_t"].double()


def _exact_dequantize(codes, scales):
    """(-1)^s 2^(e-1) (1 + m/2), or m/2 where e = 0, times 2^(S-127)."""
    N = codes.shape[0]
    c = torch.stack([codes % 16, codes // 16], -1).reshape(N, -1).double()
    sign = 1 - 2 * torch.floor(c / 8)
    mag = c % 8
    e, m = torch.floor(mag / 2), mag % 2
    v = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    scale = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return sign * v * scale


def _exact_weights(case, logits, bias):
    """Weights by repeated selection: the best expert of the groups left, k times."""
    lg = logits.double()
    T, E = lg.shape
    G, size = case["groups"], E // case["groups"]
    on = ~torch.isinf(lg)
    if case["score"] == "sigmoid":
        s = torch.sigmoid(lg)
    else:
        s = torch.exp(lg - torch.logsumexp(lg, -1, keepdim=True))
    s = torch.where(on, s, torch.zeros_like(s))
    c = s + (0 if bias is None else bias.double())
    low = torch.full_like(c, -math.inf)
    c = torch.where(on, c, low)
    if G > 1:
        by_group = c.reshape(T, G, size)
        best, at = by_group.max(-1)
        if case["group_top"] == 2:
            second = by_group.scatter(2, at.unsqueeze(-1), -math.inf).amax(-1)
            best = torch.where(torch.isinf(second), best, best + second)
        allowed = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        rows = torch.arange(T, device=c.device)
        for _ in range(case["top_groups"]):
            # the first of equal values: a running position breaks ties towards the lower index
            g = ((best == best.amax(-1, keepdim=True)) & ~allowed).int().argmax(-1)
            allowed[rows, g] = True
            best = torch.where(allowed, torch.full_like(best, -math.inf), best)
        c = torch.where(allowed.repeat_interleave(size, 1), c, low)
    picked = []
    c = c.clone()
    for _ in range(case["k"]):
        v, i = c.max(-1)
        picked.append(torch.where(torch.isinf(v), torch.zeros_like(v), s.gather(1, i[:, None])[:, 0]))
        c.scatter_(1, i[:, None], -math.inf)
    w = torch.stack(picked, -1)
    if case["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp_min(1e-300), torch.zeros_like(w))
    return w * case["scale"]
