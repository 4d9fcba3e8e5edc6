// Routing with scores for sm_100a: softmax-over-all or sigmoid scores, a bias that
// takes part in the choice only, experts in groups of which a few are kept, top-k,
// renormalised and scaled weights; then the tables of the plain routing (per-expert
// counts and offsets, the expert-sorted permutation of the pairs and its inverse).
//
// Per token of logits l [E] (definitions in include/mxfp4.h):
//   s_e = sigmoid(l_e) or exp(l_e - m) / sum exp(l - m);   c_e = s_e + b_e;
//   a group's value is the sum of its one or two largest c; the top_groups groups by
//   (value desc, index asc) are kept; the top_k experts of those by (c desc, id asc);
//   w_j = s_{id_j}, over their sum if renormalised, times scale.
// The choice is the one that 64-bit arithmetic makes, so that two experts whose scores lie a
// rounding of fp32 apart are not swapped.  It is made in fp32 with a bound on the error of c.
// Where two neighbours of the chosen order (the first one left out among them) lie closer
// than that, the candidates' c are computed again in 64 bits, a lane each, and ranked; where
// the groups on both sides of the cut do, the whole token is.
//
// Up to 128 tokens: one launch, a cluster of up to 8 CTAs with a warp per token; the CTAs exchange their
// per-expert pair counts through distributed shared memory.  More tokens: two kernels over contiguous
// chunks of them (route_chunks.h), one CTA each, the second launched while the first runs
// (programmatic dependent launch):
//   route_scored_topk   ids and weights, and the chunk's per-expert pair counts;
//   route_scored_place  every CTA sums the counts of the chunks before its own and of all (16-byte
//                       loads from L2), scans the experts, and ranks its chunk's pairs in ascending
//                       order by warp match masks.
// (One kernel with a barrier of the grid in between needs all its CTAs on the GPU at once and waits without a
// limit for those that are not; it was no faster on the device: 300 x 32 8.6 us against 7.8 so, 1237 x 90 12.3
// against 12.0, 65536 x 128 29.8 and 29.8.)
//
// What bounds it: the bytes are few (8192 x 256 fp32: 1.4 us at the copy bandwidth, 65536 x 128 bf16: 3.2).  A
// token takes some 720 warp instructions with groups and a bias and 260 without, and 30 to 290 more to place its
// pairs.  65536 tokens issue in 70% of the first kernel's cycles; 8192 in 51%, and the SMs are at work in 64% of the
// time only: what two launches and the last warps of each chunk leave open (counters of both kernels).  Times of the whole routing: 1 x 32 4.2 us, 64 x 256 in 8 groups
// 7.1, 1237 x 90 in 6 groups 12, 8192 x 256 in 8 groups 19, 65536 x 128 30 (700 GB/s).
#include "common.cuh"
#include "internal.h"
#include "route_chunks.h"

namespace mx {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
// Tokens of a cluster, a warp each, 16 to a CTA.  (256 experts in 8 groups, us: 128 tokens 8.4 and, by two kernels,
// 129 9.5; with 32 to a CTA 256 tokens 12.8, by two kernels 9.9.)
constexpr int kClusterWarps = 16;
constexpr int kClusterTokens = kMaxCluster * kClusterWarps;
constexpr int kMaxE = 256;
constexpr int kMaxChunks = kRouteMaxChunks;
constexpr uint32_t kFull = 0xFFFFFFFFu;

// A double's place in the order of the choice, larger is better: the bits folded so
// that integer order is numeric order, the two zeros equal, NaN below -inf.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return 0;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));   // -0 + 0 = +0
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// The same order on 32 bits; 0 is left for items that are not in the running.
__device__ __forceinline__ uint32_t order_key32(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 + 0 = +0
    return v != v ? 1u : (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value32(uint32_t key) {
    return __uint_as_float(key == 1u ? 0x7FC00000u : (key >> 31) ? (key & 0x7FFFFFFFu) : ~key);
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Where a token's experts live in the LT lanes that work on it: 2^seg_log2 lanes per group, `per`
// consecutive experts of it per lane (fewer, or none, at the group's end).
struct Lanes {
    int g, base, n;   // the lane's group, first expert and number of experts
    __device__ __forceinline__ Lanes(const RouteScoredArgs& a, const RouteLanes& l, int lane) {
        g = lane >> l.seg_log2;
        const int first = (lane & ((1 << l.seg_log2) - 1)) * l.per;
        base = g * a.group_size + first;
        n = g < a.n_groups ? max(0, min(l.per, a.group_size - first)) : 0;
    }
    __device__ __forceinline__ bool has(int i) const { return i < n; }
    __device__ __forceinline__ int expert(int i) const { return base + i; }
};

// Largest over the LT lanes of a token.
template <int LT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LT == 32) {
        return __reduce_max_sync(kFull, v);
    } else {
#pragma unroll
        for (int o = LT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
}

// The lane's values of a row of logits (or of the bias); -inf past its experts.  vec: every lane has NI or
// none, and they are aligned vectors.
template <bool kBf16, int NI>
__device__ __forceinline__ void load_items(const void* row, int64_t at, int n, bool vec, float* c) {
    constexpr int kBytes = NI * (kBf16 ? 2 : 4);
    uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];
    if (NI > 1 && vec) {
        const char* p = static_cast<const char*>(row) + at * (kBf16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) w[i] = 0xFF80FF80u;
        if (n > 0) {
            if (kBytes >= 16) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
                    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
                }
            } else if (kBytes == 8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                w[0] = v.x, w[kBytes >= 8 ? 1 : 0] = v.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (kBf16) c[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
            else c[i] = n > 0 ? __uint_as_float(w[i]) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) c[i] = i < n ? load_logit<kBf16>(row, at + i) : -INFINITY;
    }
}

// 64-bit arithmetic in few instructions: a launch meets this code once, cold, and fetching the
// library functions' took longer than running them (a token in 64 bits cost 10 us).
// 1 / k!, k = 0 .. 13
__device__ __constant__ double kInvFact[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                                               1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800,
                                               1.0 / 479001600, 1.0 / 6227020800.0};
// y <- e^x for V values x <= 0 at a time (they hide each other's latency): x = n ln 2 + r, |r| <= 0.35,
// Taylor's series of e^r (the term after the last is below 2^-57), ln 2 in two parts of which n
// times the first is exact (Cody and Waite).
template <int V>
__device__ __forceinline__ void exp_neg(double* x) {
    double n[V], p[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = fmax(x[v], -800.0);       // 0 from -745.2 on
        n[v] = rint(x[v] * 1.4426950408889634);
        x[v] = fma(n[v], -0x1.62e42fefp-1, x[v]);
        x[v] = fma(n[v], -0x1.473de6af278edp-34, x[v]);
        p[v] = kInvFact[13];
    }
#pragma unroll 1
    for (int k = 12; k >= 0; --k) {
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = fma(p[v], x[v], kInvFact[k]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = static_cast<int>(n[v]), h = e / 2;      // 2^e in two factors: e reaches -1155
        x[v] = p[v] * __longlong_as_double(static_cast<int64_t>(1023 + h) << 52) *
               __longlong_as_double(static_cast<int64_t>(1023 + e - h) << 52);
    }
}
// 1 / x for x >= 1 in fp32's range: Newton's steps double the digits of the hardware's reciprocal.
__device__ __forceinline__ double inv64(double x) {
    double y = 1.f / static_cast<float>(x);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) y = fma(y, fma(-x, y, 1.0), y);
    return y;
}
// What is raised to the power e for e^(l - m), m the row's largest logit, which may be infinite (then 0 at
// each that is m); NaN stays.
__device__ __forceinline__ double below(float l, float m) { return l == m ? 0.0 : static_cast<double>(l) - m; }

// What a softmax score needs of its row, in 64 bits.
struct Row64 {
    float m;
    double scale;   // 1 / sum of e^(l - m) over the row's numbers (0 for a row without any)
};
template <bool kBf16>
__device__ __forceinline__ Row64 row64(const RouteScoredArgs& a, int64_t row, int lane) {
    Row64 r = {-INFINITY, 0.0};
    if (a.by_logit || a.score != MXFP4_SCORE_SOFTMAX) return r;
    for (int e = lane; e < a.E; e += 32) r.m = fmaxf(r.m, load_logit<kBf16>(a.logits, row + e));   // NaN left out
    r.m = order_value32(__reduce_max_sync(kFull, order_key32(r.m)));
    double sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 2 * 32) {
        double z[2];
        bool in[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float l = e + 32 * v < a.E ? load_logit<kBf16>(a.logits, row + e + 32 * v) : -INFINITY;
            in[v] = l > -INFINITY;       // neither masked nor NaN
            z[v] = in[v] ? below(l, r.m) : 0.0;
        }
        exp_neg<2>(z);
#pragma unroll
        for (int v = 0; v < 2; ++v) sum += in[v] ? z[v] : 0.0;
    }
    __syncwarp();
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (sum > 0.0) r.scale = inv64(sum);   // at least 1 then
    return r;
}
// c of V experts e with logits l.
template <int V>
__device__ __forceinline__ void choice64(const RouteScoredArgs& a, const Row64& r, const float* l, const int* e, double* c) {
    if (a.by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = l[v];
        return;
    }
    const bool soft = a.score == MXFP4_SCORE_SOFTMAX;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = soft ? below(l[v], r.m) : -fabs(static_cast<double>(l[v]));
    exp_neg<V>(c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (soft) {
            c[v] *= r.scale;
        } else {   // t = e^-|l|: 1 / (1 + t), or t / (1 + t) below 0
            const double y = inv64(1.0 + c[v]);
            c[v] = l[v] < 0.f ? c[v] * y : y;
        }
        if (a.bias) c[v] += a.bias[e[v]];
        if (l[v] == -INFINITY || l[v] != l[v]) c[v] = l[v];
    }
}

// The groups that one token keeps, a bit each, by the whole warp in 64 bits.
template <bool kBf16>
__device__ __noinline__ uint32_t group_kept64(const RouteScoredArgs& a, int64_t t, int lane) {
    const Lanes L(a, a.warp, lane);
    const int64_t row = t * a.E;
    const Row64 r64 = row64<kBf16>(a, row, lane);
    const double ninf = -static_cast<double>(INFINITY);
    double t1 = ninf, t2 = ninf;
#pragma unroll 1
    for (int i = 0; L.has(i); i += 2) {
        float l[2];
        int e[2];
        double c[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            e[v] = L.expert(L.has(i + v) ? i + v : i);
            l[v] = L.has(i + v) ? load_logit<kBf16>(a.logits, row + e[v]) : -INFINITY;
        }
        choice64<2>(a, r64, l, e, c);
#pragma unroll
        for (int v = 0; v < 2; ++v) {   // NaN takes no part
            t2 = c[v] > t1 ? t1 : c[v] > t2 ? c[v] : t2;
            t1 = c[v] > t1 ? c[v] : t1;
        }
    }
    __syncwarp();
#pragma unroll 1
    for (int o = (1 << a.warp.seg_log2) >> 1; o > 0; o >>= 1) {
        const double u1 = __shfl_xor_sync(kFull, t1, o), u2 = __shfl_xor_sync(kFull, t2, o);
        t2 = fmax(fmin(t1, u1), fmax(t2, u2));
        t1 = fmax(t1, u1);
    }
    const double v = a.group_top == 2 && t2 != ninf ? t1 + t2 : t1;
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.n_groups; ++g) {
        const double u = __shfl_sync(kFull, v, g << a.warp.seg_log2);
        rank += u > v || (u == v && g < L.g);
    }
    return __reduce_or_sync(kFull, L.g < a.n_groups && rank < a.top_groups ? 1u << L.g : 0u);
}

// The chosen experts of one token whose kept groups are known, by the whole warp in 64 bits: for
// rows with NaN or infinities and for long runs of close values.  Lane j < top_k returns the
// id of slot j.
template <bool kBf16>
__device__ __noinline__ int choose64(const RouteScoredArgs& a, int64_t t, int lane, uint32_t kept) {
    const Lanes L(a, a.warp, lane);
    const bool on = L.g < 32 && ((kept >> L.g) & 1u);
    const int64_t row = t * a.E;
    const Row64 r64 = row64<kBf16>(a, row, lane);
    uint32_t live = 0;   // items that may still be chosen
    for (int i = 0; on && L.has(i); ++i) live |= 1u << i;
    __syncwarp();
    int mine = 0;
#pragma unroll 1
    for (int j = 0; j < a.top_k; ++j) {
        uint64_t best = 0;
        int id = 0x7FFFFFFF, at = 0;
#pragma unroll 1
        for (int i = 0; (live >> i) != 0; ++i) {
            if ((live >> i) & 1u) {
                const int e = L.expert(i);
                const float l = load_logit<kBf16>(a.logits, row + e);
                double c;
                choice64<1>(a, r64, &l, &e, &c);
                const uint64_t k = order_key(c);
                if (id == 0x7FFFFFFF || k > best) {   // items ascend in e: the first of equals stays
                    best = k;
                    id = e;
                    at = i;
                }
            }
        }
        __syncwarp();
        const int own = id;
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t ob = __shfl_xor_sync(kFull, best, o);
            const int oid = __shfl_xor_sync(kFull, id, o);
            if (oid != 0x7FFFFFFF && (id == 0x7FFFFFFF || ob > best || (ob == best && oid < id))) {
                best = ob;
                id = oid;
            }
        }
        if (own == id) live &= ~(1u << at);
        if (lane == j) mine = id;
    }
    return mine;
}

// The first n lanes' experts (by the whole warp; packed keys in fp32's order, at least the top_k best of the token and
// nothing nearer than fp32 tells behind them) in the exact order: lane j < top_k returns slot j.
template <bool kBf16>
__device__ __noinline__ int resolve64(const RouteScoredArgs& a, int64_t t, int lane, uint32_t packed, int n) {
    const int id = 255 - static_cast<int>(packed & 255u);
    const int64_t row = t * a.E;
    const Row64 r64 = row64<kBf16>(a, row, lane);
    const int e = lane < n ? id : 0;
    const float l = lane < n ? load_logit<kBf16>(a.logits, row + e) : -INFINITY;
    double c;
    choice64<1>(a, r64, &l, &e, &c);
    __syncwarp();
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double u = __shfl_sync(kFull, c, i);
        const int uid = __shfl_sync(kFull, id, i);
        rank += u > c || (u == c && uid < id);
    }
    int mine = 0;
    for (int i = 0; i < n; ++i) {
        const int r = __shfl_sync(kFull, rank, i), e = __shfl_sync(kFull, id, i);
        if (r == lane) mine = e;
    }
    return mine;
}

// 2^x and 1 / x in hardware: off by at most 2^-22 and 2^-23 of the result (subnormals become 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Descending, by a merge sort whose comparisons are fixed at compile time.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t* k) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1) {
#pragma unroll
        for (int q = p; q >= 1; q >>= 1) {
#pragma unroll
            for (int x = 0; x < N; ++x) {
                // Batcher's network: x and x + q meet where x lies in the first half of a block of 2 q
                // (counted from q % p) and both are in the same block of 2 p
                const int y = x + q;
                if (y < N && x >= q % p && (x - q % p) % (2 * q) < q && x / (2 * p) == y / (2 * p)) {
                    const uint32_t hi = max(k[x], k[y]), lo = min(k[x], k[y]);
                    k[x] = hi;
                    k[y] = lo;
                }
            }
        }
    }
}

// Steps of 2^-24 of the range that s + bias can have in this call; near: what rounding adds.
struct Steps {
    float lo, scale, near;
    __device__ __forceinline__ Steps(const RouteScoredArgs& a, int lane) {
        float b0 = a.bias ? INFINITY : 0.f, b1 = a.bias ? -INFINITY : 0.f;
        if (a.bias) {
            for (int e = lane; e < a.E; e += 32) {
                const float b = __ldg(a.bias + e);
                if (fabsf(b) < INFINITY) b0 = fminf(b0, b), b1 = fmaxf(b1, b);
            }
        }
        b0 = -order_value32(__reduce_max_sync(kFull, order_key32(-b0)));
        b1 = order_value32(__reduce_max_sync(kFull, order_key32(b1)));
        if (!(b0 <= b1)) b0 = b1 = 0.f;   // no finite bias
        lo = b0;
        scale = (0x1p24f - 16.f) / (1.f + (b1 - b0));
        near = fminf(0x1p-22f * (1.f + fmaxf(fabsf(b0), fabsf(b1))) * scale, 0x1p24f) + 3.f;
    }
};

// The chosen experts of token t0 + lane / LT (its lane j < top_k returns the id of slot j; past t1 there is no
// token), and for softmax scores that need them the row's maximum and sum of exp(l - m) (NaN left
// out, an infinite maximum counts 1 for each of its experts).
//
// One key per item: 24 bits that order c, then the complement of the expert's id.  Every lane sorts
// its items' keys; each round takes the largest head of the lanes' lists.  bf16 logits that order
// the choice themselves are exact in 16 of the 24 bits; fp32 ones are taken in steps of 2^-24 of
// the row's range, scores in the call's Steps.
template <bool kBf16, int NI, int LT>
__device__ __forceinline__ int choose(const RouteScoredArgs& a, const Steps& st, int64_t t0, int64_t t1, int lane,
                                      float* m_out, float* sum_out) {
    constexpr uint32_t kMine = LT == 32 ? kFull : (1u << (LT & 31)) - 1u;   // a token's lanes, from the first
    const int sub = lane / LT, at = lane % LT;
    const int64_t t = t0 + sub;
    const Lanes L(a, a.lanes, at);
    const int items = t < t1 ? L.n : 0;
    float c[NI], b[NI];
    load_items<kBf16, NI>(a.logits, t * a.E + L.base, items, a.lanes.vec, c);
    if (a.bias) load_items<false, NI>(a.bias, L.base, L.n, a.lanes.vec, b);
    else {
#pragma unroll
        for (int i = 0; i < NI; ++i) b[i] = 0.f;
    }
    // Two exact c further apart than err keep their order in fp32.  With d = l - m: exp's argument
    // is rounded (|d| 2^-23.4 of the result) and ex2 is off by 2^-22, so e^d by at most 2^-21.5
    // absolutely; the sum of at most 21 rounded additions and the quotient keep s within 2^-18 of
    // the largest score.  A sigmoid: (1 - s) s (|l| 2^-23.4 + 2^-22) for e^-l, 2^-24 s for the sum
    // and 2^-23 s for the quotient, together below 2^-21.4.
    float err = 0.f;
    if (a.score == MXFP4_SCORE_SOFTMAX) {
        if (!a.by_logit || !a.renorm) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NI; ++i) m = fmaxf(m, c[i]);
            m = order_value32(lanes_max<LT>(order_key32(m)));
            float sum = 0.f, e[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                e[i] = c[i] == -INFINITY ? 0.f : c[i] == m ? 1.f : ex2((c[i] - m) * kLog2e);
                sum += e[i] == e[i] ? e[i] : 0.f;
            }
#pragma unroll
            for (int o = LT / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            *m_out = m;
            *sum_out = sum;
            if (!a.by_logit) {
                const float inv = rcp(sum);
                err = 0x1p-17f * inv;
#pragma unroll
                for (int i = 0; i < NI; ++i) c[i] = c[i] == -INFINITY ? -INFINITY : e[i] * inv + b[i];
            }
        }
    } else if (!a.by_logit) {
        err = 0x1.8p-21f;   // twice 2^-21.4
#pragma unroll
        for (int i = 0; i < NI; ++i)
            c[i] = c[i] == -INFINITY ? -INFINITY : rcp(1.f + ex2(-kLog2e * c[i])) + b[i];
    }
    const bool exact = kBf16 && a.by_logit;
    bool close = false;   // fp32 does not tell
    bool on = true;       // the lane's group is kept
    if (a.top_groups < a.n_groups) {
        float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const float v = c[i] == c[i] ? c[i] : -INFINITY;   // NaN takes no part
            t2 = fmaxf(t2, fminf(t1, v));
            t1 = fmaxf(t1, v);
        }
        for (int o = (1 << a.lanes.seg_log2) >> 1; o > 0; o >>= 1) {
            const float u1 = __shfl_xor_sync(kFull, t1, o), u2 = __shfl_xor_sync(kFull, t2, o);
            t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
            t1 = fmaxf(t1, u1);
        }
        const float second = a.group_top == 2 && t2 != -INFINITY ? t2 : 0.f;
        const bool real = L.g < a.n_groups;
        uint32_t left = real ? order_key32(t1 + second) : 0u;   // 0 once the group is kept
        uint32_t last = 0;
        bool won = false;
#pragma unroll 1
        for (int j = 0; j < a.top_groups; ++j) {   // the best of those left, the first of equals
            last = lanes_max<LT>(left);
            const uint32_t best = (__ballot_sync(kFull, left == last) >> (sub * LT)) & kMine;
            won = L.g == (__ffs(static_cast<int>(best)) - 1) >> a.lanes.seg_log2;
            if (won) left = 0u;
        }
        on = left == 0u;
        if (!exact) {   // the last group kept and the first left out
            const uint32_t out = lanes_max<LT>(left);
            const float x = order_value32(last), y = order_value32(out);
            const float big = real && (won || left == out) ? fmaxf(fabsf(t1), fabsf(second)) : 0.f;
            const bool near = y > -INFINITY && !(x - y > 2.f * err + 0x1p-21f * big);
            const uint32_t who = __ballot_sync(kFull, near);
            for (int s = 0; who != 0u && s < 32 / LT; ++s) {
                if ((who >> (s * LT)) & kMine) {
                    const uint32_t kept = group_kept64<kBf16>(a, t0 + s, lane);
                    if (sub == s) on = L.g < 32 && ((kept >> L.g) & 1u);
                }
            }
        }
    }
    uint32_t key[NI], near = 0;   // near: keys of neighbours no further apart are close
    const int n = on ? items : 0;
    const uint32_t id0 = static_cast<uint32_t>(255 - L.base);
    if (exact) {
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = i < n ? (max(order_key32(c[i]) >> 16, 1u) << 8) + (id0 - i) : 0u;
    } else {
        float lo = st.lo, scale = st.scale;
        if (a.by_logit) {
            float x = INFINITY, y = -INFINITY;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                y = fmaxf(y, c[i]);
                x = c[i] == -INFINITY ? x : fminf(x, c[i]);
            }
            y = order_value32(lanes_max<LT>(order_key32(y)));
            lo = -order_value32(lanes_max<LT>(order_key32(-x)));
            scale = y > lo ? fminf((0x1p24f - 16.f) / (y - lo), 0x1p100f) : 0.f;
            near = 3u;    // the roundings of the difference and of the product
        } else {
            near = static_cast<uint32_t>(fminf(err * scale, 0x1p24f) + st.near);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            close |= !(c[i] < 0x1p127f);   // NaN or (nearly) infinite
            // -inf becomes 0, as close to the smallest: masked experts are ordered in 64 bits
            const uint32_t q = 4u + static_cast<uint32_t>((c[i] - lo) * scale);
            key[i] = i < n ? (q << 8) + (id0 - i) : 0u;
        }
    }
    sort_descending<NI>(key);
    uint32_t got = 0, top = 0;   // lane j of the token: the j-th best
    auto next = [&] {
        top = lanes_max<LT>(key[0]);
        const bool pop = key[0] == top;   // keys are distinct, but for the 0 of empty lists
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = pop ? (i + 1 < NI ? key[i + 1] : 0u) : key[i];
    };
    const int rounds = exact ? a.top_k : a.top_k + 1;   // one more: the first left out
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        next();
        if (at == j) got = top;
    }
    int mine = 255 - static_cast<int>(got & 255u);
    if (exact) return mine;
    const uint32_t prev = __shfl_up_sync(kFull, got, 1, LT);
    const bool tie = at > 0 && got != 0u && (prev >> 8) - (got >> 8) <= near;   // got is 0 past the rounds
    const uint32_t ties = __ballot_sync(kFull, tie), odd = __ballot_sync(kFull, close);
    if ((ties | odd) == 0u) return mine;
    // if the first left out is close, so may be those behind it: as long as one token's list goes on,
    // up to its LT-th (then the length is LT)
    int length = a.top_k;
    bool more = ((ties >> (sub * LT)) & kMine) >> length & 1u;
    uint32_t last = top;
    if (more) ++length;
    while (__any_sync(kFull, more)) {
        next();
        more = more && length < LT && top != 0u && (last >> 8) - (top >> 8) <= near;
        if (more) {
            if (at == length) got = top;
            last = top;
            ++length;
        }
    }
#pragma unroll 1
    for (int s = 0; s < 32 / LT; ++s) {   // one token after the other, by the whole warp
        const uint32_t its = kMine << (s * LT);
        if (((ties | odd) & its) == 0u) continue;
        const int many = __shfl_sync(kFull, length, s * LT);
        int ids;
        if ((odd & its) != 0u || many >= LT) {
            const uint32_t kept = __reduce_or_sync(kFull, sub == s && on && L.g < a.n_groups ? 1u << L.g : 0u);
            ids = choose64<kBf16>(a, t0 + s, lane, kept);
        } else {
            ids = resolve64<kBf16>(a, t0 + s, lane, __shfl_sync(kFull, got, s * LT + lane % LT), many);
        }
        ids = __shfl_sync(kFull, ids, at);
        if (sub == s) mine = ids;
    }
    return mine;
}

// log of the smallest 64-bit number, 2^-1074, less half a step: scores below it are 0
constexpr float kLogTiny = -745.13f;

// Slot j's weight on lane j < top_k, from its logit l.  A score that is 0 in 64 bits weighs 0 (l = -inf, or
// a mask of the type's lowest value), and so does every slot of a token whose chosen scores are all 0.
template <int LT>
__device__ __forceinline__ float slot_weight(const RouteScoredArgs& a, float l, bool on, float m, float sum) {
    const bool soft = a.score == MXFP4_SCORE_SOFTMAX;
    // (where the logits order the choice, the first chosen is the row's largest)
    if (soft && a.by_logit && a.renorm) m = __shfl_sync(kFull, l, 0, LT);
    float w = soft ? (l == m ? 1.f : expf(l - m)) : __fdividef(1.f, 1.f + expf(-l));
    if (!on || l == -INFINITY) w = 0.f;
    if (!a.renorm) return w == 0.f ? 0.f : w * (soft ? a.scale / sum : a.scale);   // (sum is 0 where all are masked)
    float s = w;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    s = __shfl_sync(kFull, s, 0, LT);
    const bool tiny = s < 0x1p-60f;
    if (__any_sync(kFull, tiny)) {   // scores so small that they lose bits (or are all 0): relative to the largest chosen
        float top = on && l == l ? l : -INFINITY;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        float v = l == top ? 1.f : expf(l - top);       // a sigmoid far below 0 is e^l
        if (!on || l == -INFINITY || l - (soft ? m : 0.f) < kLogTiny) v = 0.f;
        float u = v;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(kFull, u, o);
        if (tiny) w = v, s = u;
    }
    return s == 0.f ? 0.f : w / s * a.scale;
}

// Top-k, weights and the pair counts of tokens [t0, t1), LT lanes to a token; s_hist [E] zeroed before.
template <bool kBf16, int NI, int LT>
__device__ __forceinline__ void topk_chunk(const RouteScoredArgs& a, int64_t t0, int64_t t1, int32_t* s_hist) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kTokens = 32 / LT;   // of a warp at a time
    const Steps st(a, lane);
    for (int64_t t = t0 + warp * kTokens; t < t1; t += blockDim.x / LT) {
        float m = -INFINITY, sum = 1.f;
        const int id = choose<kBf16, NI, LT>(a, st, t, t1, lane, &m, &sum);
        const int64_t mine = t + lane / LT;
        const bool on = lane % LT < a.top_k && mine < t1;
        const float l = on ? load_logit<kBf16>(a.logits, mine * a.E + id) : -INFINITY;
        const float w = slot_weight<LT>(a, l, on, m, sum);
        if (on) {
            const int p = static_cast<int>(mine) * a.top_k + lane % LT;
            a.ids[p] = id;
            a.weights[p] = w;
            atomicAdd(&s_hist[id], 1);   // a count: its order does not matter
        }
    }
}

// Exclusive scan of s_tot [E] into s_off [E + 1] by warp 0 (8 experts per lane).
__device__ void scan_experts(const int32_t* s_tot, int32_t* s_off, int E) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int v[kMaxE / 32], run = 0;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = lane * (kMaxE / 32) + i;
            v[i] = run;
            run += e < E ? s_tot[e] : 0;
        }
        int x = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        const int base = x - run;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = lane * (kMaxE / 32) + i;
            if (e < E) s_off[e] = base + v[i];
        }
        if (lane == 31) s_off[E] = x;
    }
}

// perm and inv of pairs [p0, p1): s_base[e] is the sorted position of the range's first pair of
// expert e.  Each warp takes a run of up to kHold 32-pair strips at a time; the lanes of a strip that
// hold the same expert are one match mask.  s_cnt: [warps][kMaxE].
constexpr int kHold = 4;
__device__ __forceinline__ void place_chunk(const RouteScoredArgs& a, int64_t p0, int64_t p1, int32_t* s_base,
                                            int32_t* s_cnt) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
    const uint32_t lt = (1u << lane) - 1u;
    int32_t* cnt = s_cnt + warp * kMaxE;
    for (; p0 < p1; p0 += 32 * kHold * warps) {
        const int strips = static_cast<int>(min(static_cast<int64_t>(kHold * warps), (p1 - p0 + 31) / 32));
        const int per = (strips + warps - 1) / warps, used = (strips + per - 1) / per;   // strips a warp, warps
        int e[kHold];
        uint32_t mask[kHold];
#pragma unroll
        for (int s = 0; s < kHold; ++s) {
            const int64_t p = p0 + 32 * (per * warp + s) + lane;
            e[s] = s < per && p < p1 ? a.ids[p] : kMaxE + lane;
        }
        for (int i = threadIdx.x; i < used * (kMaxE / 4); i += blockDim.x)
            reinterpret_cast<int4*>(s_cnt)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kHold; ++s) {
            if (s < per) {
                mask[s] = __match_any_sync(kFull, e[s]);
                if (e[s] < kMaxE && (mask[s] & lt) == 0) cnt[e[s]] += __popc(mask[s]);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < a.E; x += blockDim.x) {
            int run = s_base[x];
            for (int w = 0; w < used; w += 8) {
                int v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = w + i < used ? s_cnt[(w + i) * kMaxE + x] : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (w + i < used) s_cnt[(w + i) * kMaxE + x] = run;
                    run += v[i];
                }
            }
            s_base[x] = run;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kHold; ++s) {
            if (s < per) {
                const int64_t p = p0 + 32 * (per * warp + s) + lane;
                const int first = e[s] < kMaxE ? cnt[e[s]] : 0;
                __syncwarp();
                if (e[s] < kMaxE) {
                    const int pos = first + __popc(mask[s] & lt);
                    a.perm[pos] = static_cast<int32_t>(p);
                    a.inv[p] = pos;
                    if ((mask[s] & lt) == 0) cnt[e[s]] = first + __popc(mask[s]);
                }
                __syncwarp();
            }
        }
        __syncthreads();   // the counts are used up
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int32_t ld_rank(const int32_t* p, uint32_t rank) {   // CTA rank's copy of *p
    uint32_t addr;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The whole routing of at most kClusterTokens tokens: gridDim.x CTAs, one cluster.
template <bool kBf16, int NI>
__global__ void __launch_bounds__(32 * kClusterWarps)
route_scored_cluster_kernel(const __grid_constant__ RouteScoredArgs a) {
    __shared__ int32_t s_hist[kMaxE], s_sum[kMaxE], s_base[kMaxE], s_off[kMaxE + 1];
    __shared__ __align__(16) int32_t s_cnt[kClusterWarps * kMaxE];
    for (int e = threadIdx.x; e < kMaxE; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int nb = gridDim.x, me = static_cast<int>(cluster_rank());
    const int64_t t0 = min(a.T, a.chunk * me), t1 = min(a.T, t0 + a.chunk);
    topk_chunk<kBf16, NI, 32>(a, t0, t1, s_hist);
    __syncwarp();
    cluster_barrier();   // every CTA's counts are there, and this one's ids
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int v[kMaxCluster], tot = 0, before = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) v[q] = q < nb ? ld_rank(s_hist + e, q) : 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            tot += v[q];
            before += q < me ? v[q] : 0;
        }
        s_sum[e] = tot;
        s_base[e] = before;
    }
    __syncwarp();
    cluster_barrier();   // no CTA reads another's counts any more (and this one's sums are there)
    scan_experts(s_sum, s_off, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
        if (me == 0) a.offsets[e] = s_off[e];
        if (e < a.E) {
            if (me == 0) a.counts[e] = s_sum[e];
            s_base[e] += s_off[e];
        }
    }
    __syncthreads();
    place_chunk(a, t0 * a.top_k, t1 * a.top_k, s_base, s_cnt);
}

// More tokens: a chunk of them per CTA, its ids and weights and a row of its pair counts.
template <bool kBf16, int NI, int LT>
__global__ void __launch_bounds__(kThreads)
route_scored_topk_kernel(const __grid_constant__ RouteScoredArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int32_t s_hist[kMaxE];
    for (int e = threadIdx.x; e < kMaxE; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int64_t t0 = a.chunk * blockIdx.x, t1 = min(a.T, t0 + a.chunk);
    topk_chunk<kBf16, NI, LT>(a, t0, t1, s_hist);
    __syncthreads();
    const int row = (a.E + 3) / 4 * 4;   // whole 16-byte vectors
    for (int e = threadIdx.x; e < row; e += blockDim.x) a.chunk_counts[blockIdx.x * row + e] = s_hist[e];
}

// A chunk's pairs to their places, from all chunks' counts.
__global__ void __launch_bounds__(kThreads)
route_scored_place_kernel(const __grid_constant__ RouteScoredArgs a) {
    // the threads in parts of kMaxE / 4, four experts per thread: part q sums chunks q, q + kParts, ...
    __shared__ int32_t s_off[kMaxE + 1], s_base[kMaxE], s_sum[kMaxE];
    __shared__ __align__(16) int32_t s_cnt[kWarps * kMaxE];   // first the parts' sums, then the warps' counts
    constexpr int kParts = kThreads / (kMaxE / 4), kEach = (kMaxChunks + kParts - 1) / kParts;
    static_assert(2 * kParts * kMaxE <= kWarps * kMaxE, "the parts' sums fit");
    int4(*s_tot)[kMaxE / 4] = reinterpret_cast<int4(*)[kMaxE / 4]>(s_cnt);
    int4(*s_before)[kMaxE / 4] = s_tot + kParts;
    const int nb = gridDim.x, me = blockIdx.x;
    const int e4 = threadIdx.x % (kMaxE / 4), part = threadIdx.x / (kMaxE / 4), row4 = (a.E + 3) / 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the chunks' counts and ids are complete
    if (e4 < row4) {
        int4 tot = make_int4(0, 0, 0, 0), before = tot;
        int4 v[kEach];   // all in flight
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int c = part + kParts * i;
            v[i] = c < nb ? __ldcg(reinterpret_cast<const int4*>(a.chunk_counts) + c * row4 + e4) : make_int4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            tot.x += v[i].x, tot.y += v[i].y, tot.z += v[i].z, tot.w += v[i].w;
            if (part + kParts * i < me) before.x += v[i].x, before.y += v[i].y, before.z += v[i].z, before.w += v[i].w;
        }
        s_tot[part][e4] = tot;
        s_before[part][e4] = before;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int tot = 0, before = 0;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            tot += reinterpret_cast<const int32_t*>(s_tot[q])[e];
            before += reinterpret_cast<const int32_t*>(s_before[q])[e];
        }
        s_sum[e] = tot;
        s_base[e] = before;
    }
    __syncthreads();
    scan_experts(s_sum, s_off, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
        if (me == 0) a.offsets[e] = s_off[e];
        if (e < a.E) {
            if (me == 0) a.counts[e] = s_sum[e];
            s_base[e] += s_off[e];
        }
    }
    __syncthreads();
    const int64_t t0 = a.chunk * me, t1 = min(a.T, t0 + a.chunk);
    place_chunk(a, t0 * a.top_k, t1 * a.top_k, s_base, s_cnt);
}

template <bool kBf16, int NI, int LT>
cudaError_t launch(RouteScoredArgs a, int sm_count, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (LT == 32 && a.T <= kClusterTokens) {
        const int64_t n = (a.T + kRouteMinChunk - 1) / kRouteMinChunk;
        const unsigned nc = static_cast<unsigned>(n < kMaxCluster ? n : kMaxCluster);
        a.chunk = (a.T + nc - 1) / nc;
        cfg.gridDim = dim3(nc, 1, 1);
        cfg.blockDim = dim3(32 * static_cast<unsigned>(a.chunk), 1, 1);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = nc;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, route_scored_cluster_kernel<kBf16, NI>, a);
    }
    a.chunk = route_chunk(a.T, sm_count);
    const unsigned nb = static_cast<unsigned>(route_chunks(a.T, sm_count));
    const int64_t warps = (a.chunk * LT + 31) / 32;
    route_scored_topk_kernel<kBf16, NI, LT><<<nb, 32 * static_cast<int>(warps > kWarps ? kWarps : warps), 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(nb, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, route_scored_place_kernel, a);
}

// LT lanes to a token; items per lane rounded up to a power of two, at most 16.
template <bool kBf16, int LT>
cudaError_t launch_items(const RouteScoredArgs& a, int sm_count, cudaStream_t stream) {
    if (a.lanes.per <= 1) return launch<kBf16, 1, LT>(a, sm_count, stream);
    if (a.lanes.per <= 2) return launch<kBf16, 2, LT>(a, sm_count, stream);
    if (a.lanes.per <= 4) return launch<kBf16, 4, LT>(a, sm_count, stream);
    if (a.lanes.per <= 8) return launch<kBf16, 8, LT>(a, sm_count, stream);
    return launch<kBf16, 16, LT>(a, sm_count, stream);
}

RouteLanes lanes_of(const RouteScoredArgs& a, int lt, bool bf16) {
    RouteLanes l{};
    while ((1 << l.seg_log2) < lt) ++l.seg_log2;
    while ((lt >> l.seg_log2) < a.n_groups && l.seg_log2 > 0) --l.seg_log2;
    l.per = (a.group_size + (1 << l.seg_log2) - 1) >> l.seg_log2;
    int ni = 1;
    while (ni < l.per) ni *= 2;
    const int wide = bf16 ? (ni < 8 ? ni : 8) : (ni < 4 ? ni : 4);   // elements of a lane's vector loads
    l.vec = l.per == ni && a.group_size % ni == 0 && a.E % wide == 0;
    return l;
}

}  // namespace

size_t route_scored_ws_bytes(int64_t T, int64_t E) {
    // (a device with fewer SMs has no more chunks)
    const int64_t n = route_chunks(T, kMaxChunks);
    return T <= kClusterTokens ? 0 : static_cast<size_t>(n * ((E + 3) / 4 * 4)) * sizeof(int32_t);
}

cudaError_t launch_route_scored(RouteScoredArgs a, bool bf16, int sm_count, cudaStream_t stream) {
    a.group_size = a.E / a.n_groups;
    a.warp = lanes_of(a, 32, bf16);
    // Half a warp per token where one round of warps does not hold the batch: what a token takes besides its
    // items is then shared by two (8192 x 128 11.2 -> 10.4 us, 65536 x 128 35.6 -> 29.1, 65536 x 256 in 8
    // groups 72.5 -> 68.2).  Within one round latency counts and a token has a warp (1200 x 256 in 8 groups
    // 10.5 us, in half warps 12.2).
    if (a.T > route_max_chunks(sm_count) * kWarps && a.n_groups <= 16) {
        a.lanes = lanes_of(a, 16, bf16);
        if (a.lanes.per <= 16) return bf16 ? launch_items<true, 16>(a, sm_count, stream) : launch_items<false, 16>(a, sm_count, stream);
    }
    a.lanes = a.warp;
    return bf16 ? launch_items<true, 32>(a, sm_count, stream) : launch_items<false, 32>(a, sm_count, stream);
}

}  // namespace mx
