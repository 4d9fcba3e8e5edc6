// Linear layer for many tokens: y = bf16( act(x . W^T + bias) + residual ) with W in bf16,
// on CTA pairs (tcgen05 cta_group::2).
//
// The weights are dequantized to bf16 once per call (a pass over N K 17/32 + 2 N K bytes,
// against 2 M N K operations), so that both operands of the product come by TMA and no
// warp touches them: dequantizing inside the product costs one pass per token tile.
//
// Work tile: 256 tokens x nt output columns (nt a multiple of 32 up to 256; gated: nt / 2
// gate and the same nt / 2 up features).  CTA r of the pair holds tokens 128 r .. 128 r + 127
// as the MMA's A rows and half of the columns as its B rows; the leader (r = 0) issues
// M = 256 MMAs that read both CTAs' shared memory and write 128 accumulator lanes in each.  A pair
// thus stages 16 KB of A and nt / 2 rows of B per CTA and K stage of 64, half of the B
// bytes of two single CTAs.
//
// Roles in each CTA (8 warps): warp 0 producer (its own half of both tiles; completion is
// counted on the leader's barrier), warp 1 MMA issuer (leader only), warps 4-7 epilogue (TMEM lane
// quarters), accumulators double-buffered in TMEM (2 x 256 columns).  Every wait is bounded.
#include "linear_epilogue.cuh"

namespace mx {

namespace {

using namespace linear;

constexpr int kThreads = 256;
constexpr int kBK = 64;                        // K per stage (128 bytes per row)
constexpr int kXBytes = 128 * kBK * 2;         // A rows of one CTA
constexpr int kMaxStages = 12;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kBars = 2 * kMaxStages + 2 + 2 + 1;

struct Layout {
    int stage_bytes, stages, bias_off, bar_off, misc_off, total;
};

__host__ __device__ inline Layout make_layout(int nt) {
    Layout L;
    L.stage_bytes = kXBytes + nt / 2 * kBK * 2;
    const int fixed = 4 * 256 * 4 + kBars * 8 + 16 + 1024;
    L.stages = (kSmemLimit - fixed) / L.stage_bytes;
    if (L.stages > kMaxStages) L.stages = kMaxStages;
    L.bias_off = L.stages * L.stage_bytes;
    L.bar_off = L.bias_off + 4 * 256 * 4;      // per epilogue warp: the tile's bias
    L.misc_off = L.bar_off + kBars * 8;
    L.total = L.misc_off + 16 + 1024;          // + slack for the 1024-B alignment of the base
    return L;
}

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t on_leader(const void* p) {   // the same shared address in CTA 0
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA into this CTA's shared memory, counted on a barrier of the pair's leader.
__device__ __forceinline__ void load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}
// One arrival on the barrier at this address in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

struct Ring {
    int idx = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++idx == n) {
            idx = 0;
            ph ^= 1u;
        }
    }
};

// 32 consecutive outputs of one token (columns n .. n + 31): z -> y.
template <bool kGated>
__device__ __forceinline__ void finish32(const LinearArgs& a, int64_t m, int64_t n, const uint32_t* z, const uint32_t* u,
                                         const float* bz, const float* bu, bool vec) {
    const int64_t at = m * a.n_out + n;
    const uint16_t* res = static_cast<const uint16_t*>(a.residual);
    uint16_t* y = static_cast<uint16_t*>(a.y);
    const bool whole = vec && n + 32 <= a.n_out;
    uint4 r[4];
    if (whole && res) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const uint4*>(res + at + 8 * i);
    }
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float4 b = *reinterpret_cast<const float4*>(bz + j);
        float4 o = make_float4(__uint_as_float(z[j]) + b.x, __uint_as_float(z[j + 1]) + b.y,
                               __uint_as_float(z[j + 2]) + b.z, __uint_as_float(z[j + 3]) + b.w);
        if (kGated) {
            const float4 c = *reinterpret_cast<const float4*>(bu + j);
            o.x = over_one_plus_exp(o.x, o.x) * (__uint_as_float(u[j]) + c.x);
            o.y = over_one_plus_exp(o.y, o.y) * (__uint_as_float(u[j + 1]) + c.y);
            o.z = over_one_plus_exp(o.z, o.z) * (__uint_as_float(u[j + 2]) + c.z);
            o.w = over_one_plus_exp(o.w, o.w) * (__uint_as_float(u[j + 3]) + c.w);
        } else if (a.act != MXFP4_ACT_NONE) {
            o = activate4(a.act, o, o);
        }
        v[j] = o.x, v[j + 1] = o.y, v[j + 2] = o.z, v[j + 3] = o.w;
    }
    if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* w = v + 8 * i;
            if (res) {
                const uint32_t q[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[2 * k] += bf16_lo(q[k]);
                    w[2 * k + 1] += bf16_hi(q[k]);
                }
            }
            *reinterpret_cast<uint4*>(y + at + 8 * i) =
                make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (n + j < a.n_out) {
                float w = v[j];
                if (res) w += __uint_as_float(static_cast<uint32_t>(res[at + j]) << 16);
                y[at + j] = static_cast<uint16_t>(pack_bf16(w, w));
            }
        }
    }
}

template <bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
linear_many_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                   const LinearArgs a, int nt, int m_tiles, int tiles) {
    const Layout Ly = make_layout(nt);
    const int S = Ly.stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly.bar_off);   // stage landed in both CTAs (leader's)
    uint64_t* empty = full + kMaxStages;                               // stage consumed (pair commit)
    uint64_t* accfull = empty + kMaxStages;                            // accumulators ready (pair commit)
    uint64_t* accempty = accfull + 2;                                  // drained by 8 epilogue warps (leader's)
    uint64_t* drain = accempty + 2;
    static_assert(2 * kMaxStages + 2 + 2 + 1 == kBars, "barrier block size");
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Ly.misc_off);
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Ly.misc_off + 4);
    volatile int* s_never = reinterpret_cast<volatile int*>(smem + Ly.misc_off + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int nk = static_cast<int>((a.K + kBK - 1) / kBK);
    const int cols = kGated ? nt / 2 : nt;   // output columns per tile

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], 8);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        *s_never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // both CTAs' barriers exist and TMEM is held
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        // ---------------- producer
        if (lane == 0) {
            const uint32_t full0 = on_leader(full);
            const int half = nt / 2;
            Ring c;
            int issued = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int m0 = t % m_tiles * 256 + static_cast<int>(rank) * 128;
                const int f = t / m_tiles;
                const int w0 = kGated ? static_cast<int>(rank * a.n_out) + f * half : f * nt + static_cast<int>(rank) * half;
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait(&empty[c.idx], c.ph ^ 1, s_abort)) { ok = false; break; }
                    uint8_t* dst = smem + c.idx * Ly.stage_bytes;
                    const uint32_t bar = full0 + 8 * c.idx;
                    if (rank == 0) mbar_arrive_expect_tx(&full[c.idx], 2u * Ly.stage_bytes);
                    load_pair(dst, &tmap_x, bar, i * kBK, m0);
                    load_pair(dst + kXBytes, &tmap_w, bar, i * kBK, w0);
                    c.next(S);
                    ++issued;
                }
            }
            if (!ok) {
                *s_abort = 1;
                record_status(a.status, MXFP4_ERR_TIMEOUT);
                // let the copies already issued land: the leader sees them on its barriers, the
                // other CTA waits a millisecond, far longer than a copy takes
                if (rank == 0) {
                    Ring r;
                    const int first = issued > S ? issued - S : 0;
                    for (int i = 0; i < issued; ++i) {
                        if (i >= first) mbar_wait(&full[r.idx], r.ph, s_never);
                        r.next(S);
                    }
                } else {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 1000000ull) {}
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer of the pair
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_bf16_f32(256, nt);
            Ring c;
            int lt = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
                const int b = lt & 1;
                if (!mbar_wait(&accempty[b], ((lt >> 1) & 1) ^ 1, s_abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + b * 256;
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait(&full[c.idx], c.ph, s_abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t xa = smem_u32(smem + c.idx * Ly.stage_bytes);
                    const uint64_t da = sw128_desc(xa), db = sw128_desc(xa + kXBytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j)   // 32 bytes of K per step
                        mma_pair(d, da + 2 * j, db + 2 * j, idesc, (i | j) != 0 ? 1u : 0u);
                    commit_pair(&empty[c.idx]);
                    c.next(S);
                }
                if (!ok) break;
                commit_pair(&accfull[b]);
            }
            if (!ok) {
                *s_abort = 1;
                record_status(a.status, MXFP4_ERR_TIMEOUT);
            }
            // every MMA issued by this thread completes before TMEM is released
            commit_pair(drain);
            mbar_wait(drain, 0, s_never);
        }
    } else if (warp >= 4) {
        // ---------------- epilogue: TMEM lane = token
        const int q = warp & 3;
        float* s_bias = reinterpret_cast<float*>(smem + Ly.bias_off) + q * 256;
        const uint32_t accempty0 = on_leader(accempty);
        const bool vec = a.n_out % 8 == 0;
        int lt = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
            const int64_t m = static_cast<int64_t>(t % m_tiles) * 256 + rank * 128 + q * 32 + lane;
            const int64_t n0 = static_cast<int64_t>(t / m_tiles) * cols;
            const int b = lt & 1;
            __syncwarp();
            for (int j = lane; j < nt; j += 32) {
                const int64_t n = n0 + (kGated && j >= cols ? j - cols : j);
                s_bias[j] = n < a.n_out ? bias_at(a, kGated && j >= cols ? n + a.n_out : n) : 0.f;
            }
            __syncwarp();
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&accfull[b], (lt >> 1) & 1, s_abort))) { ok = false; break; }
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * 256;
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                if (n0 + c >= a.n_out) break;
                __syncwarp();
                uint32_t z[32], u[32];
                tmem_ld_x32(base + c, z);
                if (kGated) tmem_ld_x32(base + cols + c, u);
                tmem_wait_ld();
                if (m < a.M) finish32<kGated>(a, m, n0 + c, z, u, s_bias + c, s_bias + (kGated ? cols : 0) + c, vec);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(accempty0 + 8 * b);
        }
        if (!ok) {
            *s_abort = 1;
            record_status(a.status, MXFP4_ERR_TIMEOUT);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // neither CTA's shared memory or TMEM is in use any more
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

}  // namespace

int linear_many_cols(int64_t M, int64_t n_out, bool gated, int sm_count) {
    (void)M, (void)n_out, (void)gated, (void)sm_count;
    return 256;
}

cudaError_t launch_linear_many(const LinearArgs& a, const CUtensorMap& tmap_x, const CUtensorMap& tmap_w, int nt,
                               int sm_count, cudaStream_t stream) {
    const bool gated = a.act == MXFP4_ACT_SWIGLU;
    const int cols = gated ? nt / 2 : nt;
    const int64_t m_tiles = (a.M + 255) / 256, tiles = m_tiles * ((a.n_out + cols - 1) / cols);
    if (tiles >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    const int64_t pairs = sm_count / 2 < tiles ? sm_count / 2 : tiles;
    const Layout L = make_layout(nt);
    auto kern = gated ? linear_many_kernel<true> : linear_many_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(2 * pairs), kThreads, L.total, stream>>>(tmap_x, tmap_w, a, nt, static_cast<int>(m_tiles),
                                                                         static_cast<int>(tiles));
    return cudaGetLastError();
}

}  // namespace mx
