// Linear layer for many tokens: y = bf16( act(x . W^T + bias) + residual ) with W in bf16,
// on CTA pairs (tcgen05 cta_group::2).
//
// The weights are dequantized to bf16 once per call (a pass over N K 17/32 + 2 N K bytes,
// against 2 M N K operations), so that both operands of the product come by TMA and no
// warp touches them: dequantizing inside the product costs one pass per token tile.
//
// Work tile: 256 tokens x nt accumulator columns (nt a multiple of 32 up to 256; gated: nt / 2
// gate and the same nt / 2 up features); the columns that full tiles leave are tiles of their own
// width, done last.  CTA r of the pair holds tokens 128 r .. 128 r + 127
// as the MMA's A rows and half of the columns as its B rows; the leader (r = 0) issues
// M = 256 MMAs that read both CTAs' shared memory and write 128 accumulator lanes in each.  Per 64
// of K a CTA thus stages 16 KB of A and nt / 2 rows of B, half of the B bytes of two single CTAs.
// K stages are 128 long: the issuer's and the producer's waits, once per stage, cost as much as
// two MMAs (stages of 64 took 12% longer at nt = 160).
//
// What bounds it: the MMAs of a stage (4 nt cycles) where nt = 256 and the power limit; below that
// the copies, about 47 bytes per cycle and SM from L2, so that a tile costs as 256 + nt.
//
// Measured with the weights' pass: 8192 x 2880 x 5760 gated 169 us (1609 TFLOP/s), 8192 x 2880 x 2880 100 to 121
// (1350 to 1120, residual and all), 2048 x 7680 x 2880 77 with residual (1175) and 75 without; the pass takes 12 of them.  Eight more warps that
// dequantize into shared memory inside the product, so that the pass goes, took 274, 172 and 141.
//
// Roles in each CTA (12 warps): warp 0 producer (its own half of both tiles; completion is
// counted on the leader's barrier), warp 1 MMA issuer (leader only), warps 4-11 epilogue (TMEM lane
// quarters, two warps each on alternate 16-column chunks), accumulators double-buffered in TMEM
// (2 x 256 columns).  Every wait is bounded.  An epilogue warp holds a token per lane; it passes the
// finished chunk through shared memory, so that its residual loads and its stores cover whole
// 32-byte sectors of a row, whatever the row's alignment (with a lane storing its own row, 5470 x
// 160 x 1950 took 246 us).
#include <algorithm>

#include "linear_epilogue.cuh"

namespace mx {

namespace {

using namespace linear;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStaged = 16;                    // rows of a chunk staged at a time
constexpr int kPitch = 20;                     // floats per row of a staged chunk: 16 and a conflict-free stride
constexpr int kBK = 128;                       // K per stage: two tiles of 64 (128 bytes per row)
constexpr int kXTile = 128 * 64 * 2;           // A rows of one CTA, 64 of K
constexpr int kMaxStages = 12;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kBars = 2 * kMaxStages + 2 + 2 + 1;

struct Layout {
    int stage_bytes, stages, bias_off, out_off, bar_off, misc_off, total;
};

__host__ __device__ inline Layout make_layout(int nt) {
    Layout L;
    L.stage_bytes = 2 * (kXTile + nt / 2 * 64 * 2);
    const int fixed = kEpiWarps * (128 + kStaged * kPitch) * 4 + kBars * 8 + 16 + 1024;
    L.stages = (kSmemLimit - fixed) / L.stage_bytes;
    if (L.stages > kMaxStages) L.stages = kMaxStages;
    L.bias_off = L.stages * L.stage_bytes;
    L.out_off = L.bias_off + kEpiWarps * 128 * 4;          // per epilogue warp: its columns' bias,
    L.bar_off = L.out_off + kEpiWarps * kStaged * kPitch * 4;   // and half a chunk's rows
    L.misc_off = L.bar_off + kBars * 8;
    // All of the SM's shared memory, whatever the ring takes: a CTA waits for its pair while it holds
    // TMEM, so it must not share the SM with a CTA of another cluster that may wait for TMEM.
    L.total = kSmemLimit;
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

// The launch's tiles.  Pair p of P takes the full tiles p, p + P, ... (token tile fastest, so that the
// pairs at work share weights), then, if it is one of the last narrow_pairs, every narrow_pairs-th
// narrow one.
struct Tiles {
    int nt, nt_narrow;        // accumulator columns of a full and of a narrow tile
    int m_tiles, full, narrow_pairs;
};
struct Tile {
    int m, f, nt;
};
struct Walk {
    int pair, pairs, n_full, n;
    __device__ __forceinline__ Walk(const Tiles& t) {
        pair = static_cast<int>(blockIdx.x >> 1);
        pairs = static_cast<int>(gridDim.x >> 1);
        n_full = pair < t.full ? (t.full - pair + pairs - 1) / pairs : 0;
        const int q = pair - (pairs - t.narrow_pairs);
        n = n_full + (t.narrow_pairs > 0 && q >= 0 && q < t.m_tiles ? (t.m_tiles - q + t.narrow_pairs - 1) / t.narrow_pairs : 0);
    }
    __device__ __forceinline__ Tile at(const Tiles& t, int k) const {
        if (k < n_full) {
            const int i = pair + k * pairs;
            return {i % t.m_tiles, i / t.m_tiles, t.nt};
        }
        return {pair - (pairs - t.narrow_pairs) + (k - n_full) * t.narrow_pairs, t.full / t.m_tiles, t.nt_narrow};
    }
};

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

// A chunk's way out: 32 rows (tokens) x 16 columns that start at element `at` of y, in units of `W` elements
// (8 where rows are whole 16-byte vectors, 2 where they are whole words, else 1).  Lane l takes
// units l % (16 / W) of rows l / (16 / W), + 2 W, ...; `rows` and `cols` are what the output has.
template <int W>
struct Chunk {
    static constexpr int kUnits = 16 / W, kStep = 32 / kUnits, kIters = 32 / kStep;
    __device__ __forceinline__ static void load(const uint16_t* res, int64_t at, int64_t ld, int rows, int cols, int lane,
                                                uint32_t* r) {
        const int row = lane / kUnits, col = lane % kUnits * W;
        const uint16_t* from = res + at + row * ld + col;
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            if (row + i * kStep < rows && col < cols) {
                if (W == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(from + i * kStep * ld);
                    r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
                } else if (W == 2) {
                    r[i] = *reinterpret_cast<const uint32_t*>(from + i * kStep * ld);
                } else {
                    r[i] = from[i * kStep * ld];
                }
            }
        }
    }
    // rows 16 half .. 16 half + 15 of the chunk, which are the ones staged
    __device__ __forceinline__ static void store(uint16_t* y, int64_t at, int64_t ld, int rows, int cols, int lane, int half,
                                                 const float* staged, bool add, const uint32_t* r) {
        const int row = lane / kUnits, col = lane % kUnits * W;
        uint16_t* to = y + at + (16 * half + row) * ld + col;
#pragma unroll
        for (int k = 0; k < kIters / 2; ++k) {
            const float* z = staged + (row + k * kStep) * kPitch + col;
            if (16 * half + row + k * kStep < rows && col < cols) {
                const int i = half * (kIters / 2) + k;
                if (W == 8) {
                    const float4 a = *reinterpret_cast<const float4*>(z), b = *reinterpret_cast<const float4*>(z + 4);
                    float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                    if (add) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            v[2 * x] += bf16_lo(r[4 * i + x]);
                            v[2 * x + 1] += bf16_hi(r[4 * i + x]);
                        }
                    }
                    *reinterpret_cast<uint4*>(to + k * kStep * ld) =
                        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                } else if (W == 2) {
                    float2 v = *reinterpret_cast<const float2*>(z);
                    if (add) v.x += bf16_lo(r[i]), v.y += bf16_hi(r[i]);
                    *reinterpret_cast<uint32_t*>(to + k * kStep * ld) = pack_bf16(v.x, v.y);
                } else {
                    const float v = add ? *z + bf16_lo(r[i]) : *z;
                    to[k * kStep * ld] = static_cast<uint16_t>(pack_bf16(v, v));
                }
            }
        }
    }
};

// The epilogue of one tile by one warp: the chunks c0, c0 + 32, ... of the tile's `limit` columns.
// base: this warp's TMEM lanes; bias: its chunks' (gated: the up's from 64 on).
template <bool kGated, int W>
__device__ __forceinline__ void finish_tile(const LinearArgs& a, int64_t at, int rows, int limit, int c0, int cols,
                                            uint32_t base, const float* bias, float* staged, int lane) {
    const uint16_t* res = static_cast<const uint16_t*>(a.residual);
    uint16_t* y = static_cast<uint16_t*>(a.y);
    uint32_t r[16];
    if (res && c0 < limit) Chunk<W>::load(res, at + c0, a.n_out, rows, limit - c0, lane, r);
#pragma unroll 1
    for (int c = c0; c < limit; c += 32) {
        uint32_t z[16], u[16];
        tmem_ld_x16(base + c, z);
        if (kGated) tmem_ld_x16(base + cols + c, u);
        tmem_wait_ld();
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 b = *reinterpret_cast<const float4*>(bias + (c - c0) / 2 + j);
            float4 o = make_float4(__uint_as_float(z[j]) + b.x, __uint_as_float(z[j + 1]) + b.y,
                                   __uint_as_float(z[j + 2]) + b.z, __uint_as_float(z[j + 3]) + b.w);
            if (kGated) {
                const float4 d = *reinterpret_cast<const float4*>(bias + 64 + (c - c0) / 2 + j);
                o.x = over_one_plus_exp(o.x, o.x) * (__uint_as_float(u[j]) + d.x);
                o.y = over_one_plus_exp(o.y, o.y) * (__uint_as_float(u[j + 1]) + d.y);
                o.z = over_one_plus_exp(o.z, o.z) * (__uint_as_float(u[j + 2]) + d.z);
                o.w = over_one_plus_exp(o.w, o.w) * (__uint_as_float(u[j + 3]) + d.w);
            } else if (a.act != MXFP4_ACT_NONE) {
                o = activate4(a.act, o, o);
            }
            v[j / 4] = o;
        }
        uint32_t next[16];
        if (res && c + 32 < limit) Chunk<W>::load(res, at + c + 32, a.n_out, rows, limit - c - 32, lane, next);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (lane / 16 == half) {
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(staged + (lane & 15) * kPitch + 4 * j) = v[j];
            }
            __syncwarp();
            Chunk<W>::store(y, at + c, a.n_out, rows, limit - c, lane, half, staged, res != nullptr, r);
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = next[i];
    }
}

template <bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
linear_many_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_narrow, const __grid_constant__ LinearArgs a,
                   const Tiles tiles) {
    const Layout Ly = make_layout(tiles.nt);
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
    const Walk walk(tiles);
    const int nk = static_cast<int>((a.K + kBK - 1) / kBK);
    const int full_cols = kGated ? tiles.nt / 2 : tiles.nt;   // output columns of a full tile

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        *s_never = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
        prefetch_tmap(&tmap_narrow);
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
            asm volatile("griddepcontrol.wait;" ::: "memory");   // the bf16 weights are complete
            const uint32_t full0 = on_leader(full);
            Ring c;
            int issued = 0;
            bool ok = true;
            for (int k = 0; k < walk.n && ok; ++k) {
                const Tile t = walk.at(tiles, k);
                const int m0 = t.m * 256 + static_cast<int>(rank) * 128, half = t.nt / 2;
                const int w0 = t.f * full_cols + (kGated ? static_cast<int>(rank * a.n_out) : static_cast<int>(rank) * half);
                const CUtensorMap* tw = k < walk.n_full ? &tmap_w : &tmap_narrow;
                const uint32_t bytes = 2u * 2u * (kXTile + half * 128);   // both CTAs, two tiles of 64
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait(&empty[c.idx], c.ph ^ 1, s_abort)) { ok = false; break; }
                    uint8_t* dst = smem + c.idx * Ly.stage_bytes;
                    const uint32_t bar = full0 + 8 * c.idx;
                    if (rank == 0) mbar_arrive_expect_tx(&full[c.idx], bytes);
                    load_pair(dst, &tmap_x, bar, i * kBK, m0);
                    load_pair(dst + kXTile, &tmap_x, bar, i * kBK + 64, m0);
                    load_pair(dst + 2 * kXTile, tw, bar, i * kBK, w0);
                    load_pair(dst + 2 * kXTile + half * 128, tw, bar, i * kBK + 64, w0);
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
            Ring c;
            bool ok = true;
            for (int lt = 0; lt < walk.n && ok; ++lt) {
                const int nt = walk.at(tiles, lt).nt, b = lt & 1;
                const uint32_t idesc = idesc_bf16_f32(256, nt);
                if (!mbar_wait(&accempty[b], ((lt >> 1) & 1) ^ 1, s_abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + b * 256;
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait(&full[c.idx], c.ph, s_abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t xa = smem_u32(smem + c.idx * Ly.stage_bytes);
                    const uint64_t da = sw128_desc(xa), db = sw128_desc(xa + 2 * kXTile);
                    const uint64_t next_b = static_cast<uint64_t>(nt / 2 * 128) >> 4;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {   // 32 bytes of K per step, four steps per tile
                        if (j < 4 || i * kBK + 64 < a.K)
                            mma_pair(d, da + (j & 3) * 2 + (j >> 2) * (kXTile >> 4), db + (j & 3) * 2 + (j >> 2) * next_b, idesc,
                                     (i | j) != 0 ? 1u : 0u);
                    }
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
        const int q = warp & 3, w = warp - 4;
        float* s_bias = reinterpret_cast<float*>(smem + Ly.bias_off) + w * 128;
        float* staged = reinterpret_cast<float*>(smem + Ly.out_off) + w * kStaged * kPitch;
        const uint32_t accempty0 = on_leader(accempty);
        bool ok = true;
        for (int lt = 0; lt < walk.n && ok; ++lt) {
            const Tile t = walk.at(tiles, lt);
            const int nt = t.nt, cols = kGated ? nt / 2 : nt, b = lt & 1;
            const int64_t m = static_cast<int64_t>(t.m) * 256 + rank * 128 + q * 32;
            const int64_t n0 = static_cast<int64_t>(t.f) * full_cols;
            const int rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), a.M - m)));
            const int limit = static_cast<int>(min(static_cast<int64_t>(cols), a.n_out - n0)), c0 = 16 * (w >> 2);
            __syncwarp();
            // the bias of the warp's chunks, 16 values each; gated: the gate's, then at 64 the up's
            for (int x = lane; x < 128; x += 32) {
                const int col = c0 + (kGated ? x & 63 : x) / 16 * 32 + x % 16;
                s_bias[x] = col < limit ? bias_at(a, n0 + col + (kGated && x >= 64 ? a.n_out : 0)) : 0.f;
            }
            __syncwarp();
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&accfull[b], (lt >> 1) & 1, s_abort))) { ok = false; break; }
            tc_fence_after();
            const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * 256;
            const int64_t at = m * a.n_out + n0;
            if (a.n_out % 8 == 0) finish_tile<kGated, 8>(a, at, rows, limit, c0, cols, base, s_bias, staged, lane);
            else if (a.n_out % 2 == 0) finish_tile<kGated, 2>(a, at, rows, limit, c0, cols, base, s_bias, staged, lane);
            else finish_tile<kGated, 1>(a, at, rows, limit, c0, cols, base, s_bias, staged, lane);
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

// The tiling: of the widths of a full tile, and of the ways to deal the narrow tiles out (to all pairs, or
// to those with one full tile less), the one whose longest pair is shortest, a tile counting as
// 256 + nt.  (2048 x 7680 x 2880, by nt: 256 96 us, 192 86, 160 79, 128 105.)
ManyPlan linear_many_plan(int64_t M, int64_t n_out, bool gated, int sm_count) {
    const int64_t m_tiles = (M + 255) / 256;
    ManyPlan best{};
    for (int nt = 256; nt >= 96; nt -= 32) {
        const int cols = gated ? nt / 2 : nt, unit = gated ? 16 : 32;
        const int64_t full = m_tiles * (n_out / cols);
        const int rem = static_cast<int>(n_out % cols);
        const int narrow = rem == 0 ? 0 : std::max(64, (rem + unit - 1) / unit * 32);
        const int64_t tiles = full + (narrow ? m_tiles : 0);
        const int64_t pairs = std::min<int64_t>(sm_count / 2, tiles);
        const int64_t more = full % pairs, light = pairs - more;   // pairs with one full tile more, and the others
        for (int64_t np : {light, pairs}) {
            // longest: a pair with `more` full tiles that takes narrow ones too (np == pairs), or a light one
            const int64_t each = narrow ? (m_tiles + np - 1) / np : 0, base = full / pairs;
            const int64_t heavy = (base + (more > 0)) * (256 + nt) + (np == pairs ? each * (256 + narrow) : 0);
            const int64_t cost = std::max(heavy, base * (256 + nt) + each * (256 + narrow));
            if (best.nt == 0 || cost < best.cost) best = {nt, narrow, static_cast<int>(narrow ? np : 0), pairs, full, m_tiles, cost};
        }
    }
    return best;
}

cudaError_t launch_linear_many(const LinearArgs& a, const CUtensorMap& tmap_x, const CUtensorMap& tmap_w,
                               const CUtensorMap& tmap_narrow, const ManyPlan& p, cudaStream_t stream) {
    const bool gated = a.act == MXFP4_ACT_SWIGLU;
    if (p.full + p.m_tiles >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    const Layout L = make_layout(p.nt);
    auto kern = gated ? linear_many_kernel<true> : linear_many_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
    // programmatic dependent launch: the set-up runs while the weights are still being dequantized
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * p.pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(L.total);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const Tiles t = {p.nt, p.nt_narrow, static_cast<int>(p.m_tiles), static_cast<int>(p.full), p.narrow_pairs};
    return cudaLaunchKernelEx(&cfg, kern, tmap_x, tmap_w, tmap_narrow, a, t);
}

}  // namespace mx
