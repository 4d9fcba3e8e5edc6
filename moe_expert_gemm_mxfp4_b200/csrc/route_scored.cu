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
// The choice is made on c in 64-bit arithmetic, so that two experts whose scores lie a
// rounding of fp32 apart are not swapped.
//
// Two kernels over at most kMaxChunks contiguous chunks of tokens (one CTA each):
//   route_scored_topk   one warp per token; the chunk's per-expert pair counts;
//   route_scored_place  every CTA sums the chunk counts before its own and over all
//                       (coalesced rows, from L2), scans the experts, and ranks its
//                       chunk's pairs in ascending order by warp match masks.
// A batch of one chunk does both in one launch.
#include "common.cuh"
#include "internal.h"

namespace mx {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxE = 256;
constexpr int kMaxK = 8;
constexpr int kMaxChunks = 148;    // one CTA per SM
constexpr uint32_t kFull = 0xFFFFFFFFu;

// A double's place in the order of the choice, larger is better: the bits folded so
// that integer order is numeric order, the two zeros equal, NaN below -inf.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return 0;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));   // -0 + 0 = +0
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Where expert items live in a warp: lanes in segments of `seg` (a power of two) per
// group; item i of lane r of the segment is expert r + seg * i of the group.
struct Lanes {
    int g, r, seg, gs;
    bool on;
    __device__ __forceinline__ Lanes(int lane, int n_groups, int E) {
        seg = 32;
        while (32 / seg < n_groups) seg >>= 1;
        g = lane / seg;
        r = lane % seg;
        gs = E / n_groups;
        on = g < n_groups;
    }
    __device__ __forceinline__ bool has(int i) const { return on && r + seg * i < gs; }
    __device__ __forceinline__ int expert(int i) const { return g * gs + r + seg * i; }
};

// The chosen experts of one token: lane j < top_k returns the id of slot j.  NI items
// per lane hold a whole row (E <= 256 over the lanes of n_groups segments).
template <bool kBf16, int NI>
__device__ int choose64(const RouteScoredArgs& a, int64_t t, int lane) {
    const Lanes L(lane, a.n_groups, a.E);
    double c[NI];
    uint32_t live = 0;   // items that may still be chosen
    const int64_t row = t * a.E;
    float l[NI];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        l[i] = -INFINITY;
        if (L.has(i)) {
            l[i] = load_logit<kBf16>(a.logits, row + L.expert(i));
            live |= 1u << i;
            if (l[i] > m) m = l[i];
        }
    }
    // without a bias the order of the scores is the order of the logits
    if (a.by_logit) {
#pragma unroll
        for (int i = 0; i < NI; ++i) c[i] = l[i];
    } else {
        double sum = 1.0;
        if (a.score == MXFP4_SCORE_SOFTMAX) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            sum = 0.0;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const double d = l[i];
            if (a.score == MXFP4_SCORE_SOFTMAX) {
                c[i] = l[i] == -INFINITY ? 0.0 : l[i] == m ? 1.0 : exp(d - m);
                if (c[i] == c[i]) sum += c[i];
            } else {
                c[i] = 1.0 / (1.0 + exp(-d));
            }
        }
        if (a.score == MXFP4_SCORE_SOFTMAX) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (L.has(i)) {
                const double b = a.bias ? a.bias[L.expert(i)] : 0.f;
                c[i] = l[i] == -INFINITY ? -static_cast<double>(INFINITY) : c[i] / sum + b;
            }
        }
    }
    if (a.n_groups > 1) {
        const double ninf = -static_cast<double>(INFINITY);
        double t1 = ninf, t2 = ninf;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (L.has(i) && c[i] == c[i]) {
                t2 = c[i] > t1 ? t1 : (c[i] > t2 ? c[i] : t2);
                t1 = c[i] > t1 ? c[i] : t1;
            }
        }
        for (int o = L.seg >> 1; o > 0; o >>= 1) {
            const double u1 = __shfl_xor_sync(kFull, t1, o), u2 = __shfl_xor_sync(kFull, t2, o);
            t2 = fmax(fmin(t1, u1), fmax(t2, u2));
            t1 = fmax(t1, u1);
        }
        const double v = a.group_top == 2 && t2 != ninf ? t1 + t2 : t1;
        int rank = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double u = __shfl_sync(kFull, v, g * L.seg);
            rank += u > v || (u == v && g < L.g);
        }
        if (rank >= a.top_groups) live = 0;
    }
    int mine = 0;
    for (int j = 0; j < a.top_k; ++j) {
        uint64_t best = 0;
        int id = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if ((live >> i) & 1u) {
                const uint64_t k = order_key(c[i]);
                const int e = L.expert(i);
                if (id == 0x7FFFFFFF || k > best) {   // items ascend in e: the first of equals stays
                    best = k;
                    id = e;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t ob = __shfl_xor_sync(kFull, best, o);
            const int oid = __shfl_xor_sync(kFull, id, o);
            if (oid != 0x7FFFFFFF && (id == 0x7FFFFFFF || ob > best || (ob == best && oid < id))) {
                best = ob;
                id = oid;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (L.has(i) && L.expert(i) == id) live &= ~(1u << i);
        if (lane == j) mine = id;
    }
    return mine;
}

// max and sum of exp(l - max) over the row's numbers (NaN left out, an infinite
// maximum counts 1 for each of its experts)
template <bool kBf16, int NI>
__device__ __forceinline__ void row_softmax(const RouteScoredArgs& a, int64_t t, int lane, float* m_out, float* sum_out) {
    float l[NI];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.E ? load_logit<kBf16>(a.logits, t * a.E + e) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const float z = l[i] == -INFINITY ? 0.f : l[i] == m ? 1.f : expf(l[i] - m);
        if (z == z) sum += z;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    *m_out = m;
    *sum_out = sum;
}

// log of the smallest 64-bit number, 2^-1074, less half a step: scores below it are 0
constexpr float kLogTiny = -745.13f;

// Slot j's weight on lane j < top_k, from its logit l.  Renormalised weights are taken
// relative to the largest chosen logit, so that rows of very small scores keep their
// precision.  A score that is 0 in 64 bits weighs 0 (l = -inf, or a mask of the type's
// lowest value), and so does every slot of a token whose chosen scores are all 0.
__device__ __forceinline__ float slot_weight(const RouteScoredArgs& a, float l, bool on, float m, float sum, int lane) {
    float w = 0.f;
    if (a.renorm) {
        float top = on && l == l ? l : -INFINITY;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        const float ref = a.score == MXFP4_SCORE_SOFTMAX ? m : 0.f;
        if (on && l != -INFINITY && !(l - ref < kLogTiny)) {
            if (a.score == MXFP4_SCORE_SOFTMAX) w = l == top ? 1.f : expf(l - top);
            else if (top < 0.f) w = (l == top ? 1.f : expf(l - top)) / (1.f + expf(l));
            else w = 1.f / (1.f + expf(-l));
        }
        float s = w;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        w = s == 0.f ? 0.f : w / s;
    } else if (on && l != -INFINITY) {
        w = a.score == MXFP4_SCORE_SOFTMAX ? (l == m ? 1.f : expf(l - m)) / sum : 1.f / (1.f + expf(-l));
    }
    return w * a.scale;
}

// Top-k, weights and the pair counts of tokens [t0, t1); s_hist [E] zeroed before.
template <bool kBf16, int NI>
__device__ void topk_chunk(const RouteScoredArgs& a, int64_t t0, int64_t t1, int32_t* s_hist) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = t0 + warp; t < t1; t += kWarps) {
        const int id = choose64<kBf16, NI>(a, t, lane);
        float m = 0.f, sum = 1.f;
        if (a.score == MXFP4_SCORE_SOFTMAX) row_softmax<kBf16, 8>(a, t, lane, &m, &sum);
        const bool on = lane < a.top_k;
        const float l = on ? load_logit<kBf16>(a.logits, t * a.E + id) : -INFINITY;
        const float w = slot_weight(a, l, on, m, sum, lane);
        if (on) {
            a.ids[t * a.top_k + lane] = id;
            a.weights[t * a.top_k + lane] = w;
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

// perm and inv of pairs [p0, p1): s_base[e] is the sorted position of the range's
// first pair of expert e.  Each warp takes a contiguous run of 32-pair strips; the
// lanes of a strip that hold the same expert are one match mask.  s_cnt: [kWarps][kMaxE].
__device__ void place_chunk(const RouteScoredArgs& a, int64_t p0, int64_t p1, const int32_t* s_base, int32_t* s_cnt) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * kMaxE; i += kThreads) s_cnt[i] = 0;
    __syncthreads();
    const int64_t strips = (p1 - p0 + 31) / 32;
    const int64_t s0 = strips * warp / kWarps, s1 = strips * (warp + 1) / kWarps;
    int32_t* cnt = s_cnt + warp * kMaxE;
    const uint32_t lt = (1u << lane) - 1u;
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t p = p0 + 32 * s + lane;
        const int e = p < p1 ? a.ids[p] : kMaxE + lane;
        const uint32_t mask = __match_any_sync(kFull, e);
        if (p < p1 && (mask & lt) == 0) cnt[e] += __popc(mask);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        int run = s_base[e];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int v = s_cnt[w * kMaxE + e];
            s_cnt[w * kMaxE + e] = run;
            run += v;
        }
    }
    __syncthreads();
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t p = p0 + 32 * s + lane;
        const int e = p < p1 ? a.ids[p] : kMaxE + lane;
        const uint32_t mask = __match_any_sync(kFull, e);
        const int first = p < p1 ? cnt[e] : 0;
        __syncwarp();
        if (p < p1) {
            const int pos = first + __popc(mask & lt);
            a.perm[pos] = static_cast<int32_t>(p);
            a.inv[p] = pos;
            if ((mask & lt) == 0) cnt[e] = first + __popc(mask);
        }
        __syncwarp();
    }
}

template <bool kBf16, int NI>
__global__ void __launch_bounds__(kThreads)
route_scored_one_kernel(const RouteScoredArgs a) {
    __shared__ int32_t s_hist[kMaxE], s_off[kMaxE + 1], s_cnt[kWarps * kMaxE];
    for (int e = threadIdx.x; e < kMaxE; e += kThreads) s_hist[e] = 0;
    __syncthreads();
    topk_chunk<kBf16, NI>(a, 0, a.T, s_hist);
    __syncthreads();   // the ids written above are read back below
    scan_experts(s_hist, s_off, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += kThreads) {
        a.offsets[e] = s_off[e];
        if (e < a.E) a.counts[e] = s_hist[e];
    }
    place_chunk(a, 0, a.T * a.top_k, s_off, s_cnt);
}

template <bool kBf16, int NI>
__global__ void __launch_bounds__(kThreads)
route_scored_topk_kernel(const RouteScoredArgs a) {
    __shared__ int32_t s_hist[kMaxE];
    for (int e = threadIdx.x; e < kMaxE; e += kThreads) s_hist[e] = 0;
    __syncthreads();
    const int64_t t0 = a.T * blockIdx.x / gridDim.x, t1 = a.T * (blockIdx.x + 1) / gridDim.x;
    topk_chunk<kBf16, NI>(a, t0, t1, s_hist);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.chunk_counts[blockIdx.x * a.E + e] = s_hist[e];
}

__global__ void __launch_bounds__(kThreads)
route_scored_place_kernel(const RouteScoredArgs a) {
    __shared__ int32_t s_tot[2][kMaxE], s_before[2][kMaxE], s_off[kMaxE + 1], s_cnt[kWarps * kMaxE];
    static_assert(kThreads == 2 * kMaxE, "two threads per expert");
    const int e = threadIdx.x & (kMaxE - 1), half = threadIdx.x / kMaxE;
    const int nb = gridDim.x, me = blockIdx.x;
    if (e < a.E) {
        int tot = 0, before = 0;
#pragma unroll 8
        for (int c = half; c < nb; c += 2) {
            const int v = a.chunk_counts[c * a.E + e];
            tot += v;
            if (c < me) before += v;
        }
        s_tot[half][e] = tot;
        s_before[half][e] = before;
    }
    __syncthreads();
    if (threadIdx.x < a.E) s_tot[0][e] += s_tot[1][e];
    __syncthreads();
    scan_experts(s_tot[0], s_off, a.E);
    __syncthreads();
    if (me == 0) {
        for (int i = threadIdx.x; i <= a.E; i += kThreads) {
            a.offsets[i] = s_off[i];
            if (i < a.E) a.counts[i] = s_tot[0][i];
        }
    }
    if (threadIdx.x < a.E) s_before[0][e] += s_before[1][e] + s_off[e];
    __syncthreads();
    const int64_t t0 = a.T * me / nb, t1 = a.T * (me + 1) / nb;
    place_chunk(a, t0 * a.top_k, t1 * a.top_k, s_before[0], s_cnt);
}

// Chunks of a batch: a warp per token while the SMs last, then one CTA per SM.
int64_t chunks_of(int64_t T) {
    const int64_t n = (T + kWarps - 1) / kWarps;
    return n < kMaxChunks ? n : kMaxChunks;
}

template <bool kBf16, int NI>
cudaError_t launch(const RouteScoredArgs& a, cudaStream_t stream) {
    const unsigned nb = static_cast<unsigned>(chunks_of(a.T));
    if (nb == 1) {
        route_scored_one_kernel<kBf16, NI><<<1, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    route_scored_topk_kernel<kBf16, NI><<<nb, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    route_scored_place_kernel<<<nb, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t route_scored_ws_bytes(int64_t T, int64_t E) {
    const int64_t n = chunks_of(T);
    return n == 1 ? 0 : static_cast<size_t>(n * E) * sizeof(int32_t);
}

cudaError_t launch_route_scored(const RouteScoredArgs& a, bool bf16, cudaStream_t stream) {
    // items per lane: 8 hold E <= 256 over whole-warp or power-of-two segments, 16 any group count
    int seg = 32;
    while (32 / seg < a.n_groups) seg >>= 1;
    const int items = (a.E / a.n_groups + seg - 1) / seg;
    if (items <= 8) return bf16 ? launch<true, 8>(a, stream) : launch<false, 8>(a, stream);
    return bf16 ? launch<true, 16>(a, stream) : launch<false, 16>(a, stream);
}

}  // namespace mx
