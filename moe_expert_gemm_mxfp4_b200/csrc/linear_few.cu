// Linear layer for few tokens: y = bf16( act(x . W^T + bias) + residual ) with the MXFP4
// weights fed to the tensor core as they are (tcgen05 kind::mxf8f6f4, block scales).
//
// With few tokens the weights' bytes bound the call, and turning codes into bf16 costs more
// than reading them.  So the weights stay E2M1 with their E8M0 scales (the MMA's A side),
// and the bf16 activations become two E4M3 parts with block scales (the B side):
//   x = 2^s (hi + 2^-5 lo),   2^7 <= max |x| / 2^s < 2^8 over a 32-block,
//   hi = e4m3(x / 2^s),       lo = e4m3(2^5 (x / 2^s - hi)).
// bf16 has 8 significant bits, hi takes 4, and what is left of an element fits the 4 of lo: the
// sum is exact for every element within 2^14 of its block's largest, and off by at most
// 2^-22 of that largest for the others, about what one addition in fp32 rounds.  Products with
// E2M1 are exact, sums are fp32.  A block that holds Inf or NaN gets the scale NaN, and
// hi alone passes fp32's range where x is in the last 3% of it (significands from 0xF8 on round up to
// 2^128); so a sum that is not finite is computed again from x and W themselves, and infinities
// act as in the formula.
//
// Two launches, the second overlapping the first (programmatic dependent launch):
//   linear_few_prepare  x -> hi and lo tiles in the tensor core's shared-memory image, their
//                       scales and the weights' scales in its scale-factor layout;
//   linear_few          one CTA per (128 weight rows, K range, token tile).
// Up to 16 tokens the spreading warps prepare their CTA's own part instead, and there is one
// launch: every CTA of a K range then splits the same activations, a few per lane.
// Roles (12 warps, one CTA per SM): warp 11 streams packed codes (TMA, 128 bytes per row) into a ring of
// their own; warps 0-7 spread them over the 16-element containers that the tensor core takes (8
// bytes of codes, 8 of padding), three instructions per 16 bytes; warp 8 bulk-copies
// the prepared tiles; warp 9 issues scale copies and MMAs.  A stage is 256 of K (two tiles of
// 128 containers): the waits and fences, once per stage, cost as much as its MMAs.  The CTAs of a cluster split K and sum
// their partial results through distributed shared memory in rank order (the same on every
// run); each finishes a share of the tokens.
//
// What bounds it: up to a hundred tokens neither bytes nor MMAs but the chain of a launch (set-up, the first
// codes, the spreading of a stage, the cluster's sums): 1 x 2880 x 2880 7.5 to 7.9 us (0.7 at the copy bandwidth),
// 64 x 2880 x 5760 gated 12.8 (1.5); with long weights the spreading, 32 x 7680 x 11520 28 us (1.7 TB/s); with
// several token tiles the MMAs (of both parts) and the finish, 512 x 2880 x 2880 18.3 us (464 TFLOP/s; with
// SiLU 20).
//
// hi and lo rows lie next to each other in one MMA of N = 2 Mp columns while that fits the 128
// rows of a scale atom (an MMA of N <= 64 costs the same whatever its N), else they are
// two MMAs of N = Mp into the same accumulator.
#include <atomic>

#include "linear_epilogue.cuh"

namespace mx {

namespace {

using namespace linear;

constexpr int kThreads = 384;
constexpr int kSpreadWarps = 8;
constexpr int kPrepareThreads = 256;
constexpr int kBM = 128;             // weight rows per tile
constexpr int kRow = 128;            // bytes of a row of a tile: 128 one-byte containers, half a stage of K
constexpr int kATile = kBM * kRow;
constexpr int kAtom = 512;           // scale atom: 128 rows x 4 scales
constexpr int kMaxMp = 112;          // tokens per tile: two stages and two code slots still fit
constexpr int kOwnMp = 16;           // largest token tile that is prepared where it is used: one launch instead of two
                                     // (2880 x 2880, us, called by a host 11 instead of 15; replayed from a graph 7.5 and
                                     // 7.9 for 1 token, 8.5 and 8.1 for 8, 10.2 and 8.2 for 16, where the splitting shows),
constexpr int kOwnStages = 3;        // and the stages of a CTA it is loaded ahead for
constexpr int kMaxStages = 3;
constexpr int kCodeBytes = kBM * 128;   // a code slot: a stage's 128 bytes of each row
constexpr int kMaxSlots = 6;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSms = 148;            // what the launch geometry aims at
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 256, kSfCol = 128;   // D [0, 128), scale sets of 16 columns behind it

__device__ __forceinline__ uint32_t ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
// One lane of the (converged) warp; what it issues keeps its operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// D[tmem] (+)= (A . 2^SFA) (B . 2^SFB)^T, one scale per 32 elements of K, K = 32.
__device__ __forceinline__ void mma_mxf8f6f4(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
}
// Instruction descriptor of kind::mxf8f6f4: B scale id (bits 4-5), A format E2M1 = 5 (bits 7-9),
// B format E4M3 = 0 (bits 10-12), N >> 3 (bits 17-22), scales E8M0 (bit 23), M >> 7 (bits
// 27-28), A scale id (bits 29-30).
__device__ __forceinline__ uint32_t idesc_mxf8(int N, uint32_t sf_id) {
    return (sf_id << 4) | (5u << 7) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (1u << 27) | (sf_id << 29);
}

// hi and lo of two scaled values: packed E4M3 bytes (low byte first).
__device__ __forceinline__ void split2(float a, float b, float up, uint32_t& hi, uint32_t& lo) {
    uint16_t h, l;
    uint32_t back;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
    float ha, hb;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
        : "=f"(ha), "=f"(hb) : "r"(back));
    const float ra = (a - ha) * up, rb = (b - hb) * up;   // exact: the difference has at most 5 bits
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"(rb), "f"(ra));
    hi = h;
    lo = l;
}

// Four elements of a 32-block held by 8 lanes: their parts as four E4M3 bytes each, and the block's
// scale bytes.  A block with Inf or NaN gets the scale NaN, and NaN elements.
struct Parts {
    uint32_t hi, lo, s_hi, s_lo;
};
__device__ __forceinline__ Parts split4(uint2 v) {
    // bf16 magnitudes order as integers, infinities and NaN last
    uint32_t amax = max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const bool odd = amax >= 0x7F80u;
    const int e = static_cast<int>(amax >> 7);          // biased exponent of the largest
    const int s_hi = e > 7 ? e - 7 : 0, s_lo = s_hi > 5 ? s_hi - 5 : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(254 - s_hi) << 23);   // 2^(127 - s_hi)
    const float up = __uint_as_float(static_cast<uint32_t>(127 + s_hi - s_lo) << 23);
    uint32_t h0, h1, l0, l1;
    split2(bf16_lo(v.x) * down, bf16_hi(v.x) * down, up, h0, l0);
    split2(bf16_lo(v.y) * down, bf16_hi(v.y) * down, up, h1, l1);
    Parts p;
    p.hi = odd ? 0x7F7F7F7Fu : h0 | h1 << 16;
    p.lo = odd ? 0u : l0 | l1 << 16;
    p.s_hi = odd ? 255u : static_cast<uint32_t>(s_hi);
    p.s_lo = odd ? 255u : static_cast<uint32_t>(s_lo);
    return p;
}
// Byte offset of elements 4 lane .. 4 lane + 3 of a row in a swizzled tile, and of scale j of a row in
// its atom.
__device__ __forceinline__ int tile_at(int row, int lane) {
    return row * kRow + (((lane >> 2) ^ (row & 7)) << 4) + 4 * (lane & 3);
}
__device__ __forceinline__ int atom_at(int row, int j) { return 16 * (row & 31) + 4 * (row >> 5) + j; }

struct Plan {
    int mp;            // token rows of a tile (padded to 8 or a multiple of 16)
    int t_tiles;       // token tiles of mp rows
    int own;           // the product's CTAs prepare their own part
    int stacked;       // hi and lo rows in one MMA of N = 2 mp
    int w_tiles;       // tiles of 128 weight rows
    int nk;            // K stages
    int sfb_bytes;     // scale atoms of half a stage's activations
    int b_bytes;       // prepared bytes per token tile and stage: both halves' hi and lo rows, then their scale atoms
    int stage_bytes;
    int stages;        // ring of stages (containers, activations, scales)
    int slots;         // ring of packed codes
};

// First weight row of a tile's row r, or -1 past the end.  Gated tiles hold 64 gate rows and
// the 64 up rows of the same features.
template <bool kGated>
__device__ __forceinline__ int64_t weight_row(const LinearArgs& a, int64_t f, int r) {
    if (!kGated) {
        const int64_t n = f * kBM + r;
        return n < a.N ? n : -1;
    }
    const int64_t n = f * 64 + (r & 63);
    return n < a.n_out ? n + (r >= 64 ? a.n_out : 0) : -1;
}

// ---------------------------------------------------------------- prepare
// The first 4 w_tiles CTAs lay the weights' scales out, 32 rows each: per tile and half stage an atom of
// 512 bytes, scale j of row r at byte 16 (r % 32) + 4 (r / 32) + j.  The others take (token, half
// stage) items, one per warp: 4 elements per lane, 8 lanes to a block.
template <bool kGated>
__global__ void __launch_bounds__(kPrepareThreads)
linear_few_prepare_kernel(const LinearArgs a, const Plan p, uint8_t* __restrict__ ws_b, uint8_t* __restrict__ ws_sfa) {
    grid_launch_dependents();
    extern __shared__ __align__(16) uint8_t s_rows[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kb = static_cast<int>(a.K / 32), halves = (kb + 3) / 4;
    const int w_ctas = 4 * p.w_tiles;
    if (static_cast<int>(blockIdx.x) < w_ctas) {
        // 32 rows of a tile: one run of bytes, brought over in 16-byte vectors
        const int64_t f = blockIdx.x / 4;
        const int q = blockIdx.x % 4;
        const int64_t row0 = kGated ? f * 64 + 32 * (q & 1) : f * kBM + 32 * q;
        const int64_t left = (kGated ? a.n_out : a.N) - row0;
        const int rows = left < 0 ? 0 : left > 32 ? 32 : static_cast<int>(left), len = rows * kb;
        const uint8_t* src = a.scales + (row0 + (kGated && q >= 2 ? a.n_out : 0)) * kb;
        const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
        uint8_t* dst = s_rows + shift;
        const int head = min(len, (16 - shift) & 15), body = (len - head) / 16;
#pragma unroll 4
        for (int i = tid; i < body; i += kPrepareThreads)
            reinterpret_cast<uint4*>(dst + head)[i] = __ldg(reinterpret_cast<const uint4*>(src + head) + i);
        for (int i = tid; i < head; i += kPrepareThreads) dst[i] = src[i];
        for (int i = head + 16 * body + tid; i < len; i += kPrepareThreads) dst[i] = src[i];
        __syncthreads();
        for (int j = warp; j < halves; j += kPrepareThreads / 32) {
            uint32_t w = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                w |= (lane < rows && 4 * j + b < kb ? dst[lane * kb + 4 * j + b] : 0x7Fu) << (8 * b);
            *reinterpret_cast<uint32_t*>(ws_sfa + (f * 2 * p.nk + j) * kAtom + 16 * lane + 4 * q) = w;
        }
        return;
    }
    // 32 bits hold the items: this engine takes at most kSms tiles of kMaxMp tokens, and K of 64 half stages
    const unsigned items = static_cast<unsigned>(a.M) * halves, step = (gridDim.x - w_ctas) * (kPrepareThreads / 32);
    for (unsigned it = (blockIdx.x - w_ctas) * (kPrepareThreads / 32) + warp; it < items; it += step) {
        const unsigned t = it / halves, tt = t / static_cast<unsigned>(p.mp);
        const int j = static_cast<int>(it - t * halves), r = static_cast<int>(t - tt * p.mp);
        const int k = j * kRow + 4 * lane;
        uint2 v = make_uint2(0u, 0u);
        if (k < a.K) v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + t * a.K + k));
        const Parts q = split4(v);
        uint8_t* blk = ws_b + (static_cast<int64_t>(tt) * p.nk + (j >> 1)) * p.b_bytes;
        uint8_t* tile = blk + (j & 1) * 2 * p.mp * kRow;
        const int r_lo = p.mp + r;
        *reinterpret_cast<uint32_t*>(tile + tile_at(r, lane)) = q.hi;
        *reinterpret_cast<uint32_t*>(tile + tile_at(r_lo, lane)) = q.lo;
        if ((lane & 7) == 0) {
            uint8_t* atom = blk + 4 * p.mp * kRow + (j & 1) * p.sfb_bytes;
            atom[atom_at(r, lane >> 3)] = static_cast<uint8_t>(q.s_hi);
            atom[p.stacked ? atom_at(r_lo, lane >> 3) : kAtom + atom_at(r, lane >> 3)] = static_cast<uint8_t>(q.s_lo);
        }
    }
}

// One output's sum from x and W themselves: in 64 bits, whose range no product and no partial sum leaves.  Eight
// elements a load: one thread walks all of K, and a padded batch may hold many rows with NaN
// (512 x 2880 x 2880, every row with a NaN: 4.6 ms a call; with loads of single elements 17.9).
__device__ __noinline__ float dot_direct(const LinearArgs& a, int64_t m, int64_t row) {
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.K);
    const uint32_t* c = reinterpret_cast<const uint32_t*>(a.codes + row * (a.K / 2));
    const uint8_t* scales = a.scales + row * (a.K / 32);
    const int n = static_cast<int>(a.K / 8);
    double acc = 0.0;
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
        const uint4 v = __ldg(x + i);
        const uint32_t xs[4] = {v.x, v.y, v.z, v.w}, codes = __ldg(c + i);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum = fma(static_cast<double>(bf16_lo(xs[j])), static_cast<double>(e2m1_f32((codes >> (8 * j)) & 15u)), sum);
            sum = fma(static_cast<double>(bf16_hi(xs[j])), static_cast<double>(e2m1_f32((codes >> (8 * j + 4)) & 15u)), sum);
        }
        acc = fma(sum, static_cast<double>(e8m0_f32(scales[i / 4])), acc);
    }
    return static_cast<float>(acc);
}

// ---------------------------------------------------------------- product
// SPLIT: CTAs of a cluster along K.  kOwn: the CTA prepares its activations and scales itself.
template <bool kGated, int SPLIT, bool kOwn>
__global__ void __launch_bounds__(kThreads)
linear_few_kernel(const __grid_constant__ CUtensorMap tmap_codes, const __grid_constant__ LinearArgs a, const Plan p,
                  const uint8_t* __restrict__ ws_b, const uint8_t* __restrict__ ws_sfa) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done[1];
    __shared__ uint64_t code_full[kMaxSlots], code_empty[kMaxSlots];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort, s_never;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int NS = p.stages, CS = p.slots;
    const int rank = SPLIT > 1 ? static_cast<int>(ctarank()) : 0;
    const int64_t f = blockIdx.x / SPLIT;
    const int64_t tt = blockIdx.y;
    const int64_t t0 = tt * p.mp;
    const int mt = static_cast<int>(min(static_cast<int64_t>(p.mp), a.M - t0));   // the tile's tokens
    // this CTA's K stages [j0, j0 + n); the launch keeps SPLIT <= nk, so n >= 1
    const int j0 = rank * p.nk / SPLIT;
    const int n = (rank + 1) * p.nk / SPLIT - j0;
    const int k_left = static_cast<int>(a.K) - 256 * j0;   // of K from the CTA's first element on
    constexpr int kFeat = kGated ? 64 : kBM;     // output features of the tile
    uint8_t* codes = smem + NS * p.stage_bytes;  // the code slots lie behind the stages

    // code slot i % CS <- stage i (past K: zero fill)
    auto load_codes = [&](int i) {
        uint8_t* dst = codes + i % CS * kCodeBytes;
        uint64_t* bar = &code_full[i % CS];
        const int x = 128 * (j0 + i);
        mbar_arrive_expect_tx(bar, kCodeBytes);
        tma_load_2d(dst, &tmap_codes, bar, x, static_cast<int>(f * kFeat));
        if (kGated) tma_load_2d(dst + kCodeBytes / 2, &tmap_codes, bar, x, static_cast<int>(a.n_out + f * kFeat));
    };
    if (tid == 11 * 32) {
        for (int s = 0; s < kMaxSlots; ++s) {
            mbar_init(&code_full[s], 1);
            mbar_init(&code_empty[s], kSpreadWarps);
        }
        fence_mbar_init();
        // the first copies start before the other warps are ready
        for (int i = 0; i < min(n, CS); ++i) load_codes(i);
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&full[s], kSpreadWarps + (kOwn ? 0 : 1));   // and the copies of warp 8
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        s_abort = 0;
        s_never = 0;
        fence_mbar_init();
    }
    if (warp == 10) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    // kOwn: spreading warp 4 h + w splits tokens w, w + 4, ... (at most 16) of half h of each stage and
    // fetches the scales of its rows 32 w .. 32 w + 31; all stages' are on their way from the start
    uint2 xv[kOwn ? kOwnStages : 1][4];
    uint32_t sv[kOwn ? kOwnStages : 1][4];
    if (kOwn && warp < kSpreadWarps) {
        const int kb = static_cast<int>(a.K / 32), half = warp >> 2;
        const int64_t row = weight_row<kGated>(a, f, 32 * (warp & 3) + lane);
        const uint8_t* scales = a.scales + (row < 0 ? 0 : row) * kb;
#pragma unroll
        for (int i = 0; i < kOwnStages; ++i) {
            const int64_t k = 256LL * (j0 + i) + 128 * half + 4 * lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = (warp & 3) + 4 * q, x = 8 * (j0 + i) + 4 * half + q;
                xv[i][q] = make_uint2(0u, 0u);
                if (i < n && t < mt && k < a.K)
                    xv[i][q] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + (t0 + t) * a.K + k));
                sv[i][q] = i < n && x < kb ? __ldg(scales + x) : 0x7Fu;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp < kSpreadWarps) {
        // ---------------- codes -> containers: warps 0-3 the first half of a stage, 4-7 the second; 16
        // bytes of codes of a row are containers 2 ch and 2 ch + 1, swizzled within the row's 128 bytes
        const int half = warp >> 2, ch = tid & 3, r = (tid & 127) >> 2;
        const uint32_t from = smem_u32(codes) + r * 128 + half * 64 + 16 * ch;
        const uint32_t to = smem_u32(smem) + half * kATile + r * kRow + (((2 * ch) ^ (r & 7)) << 4);
        bool ok = true;
        auto spread = [&](int i) {
            bool got = i < NS || wait_poll(&empty[i % NS], ((i / NS) & 1) ^ 1, &s_abort);
            if (got) got = wait_poll(&code_full[i % CS], (i / CS) & 1, &s_abort);
            if (!__all_sync(0xFFFFFFFFu, got)) return false;
            const uint32_t src = from + i % CS * kCodeBytes, dst = to + i % NS * p.stage_bytes;
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = lds128(src + q * 32 * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                sts64(dst + q * 32 * kRow, v[q].x, v[q].y);
                sts64((dst ^ 16u) + q * 32 * kRow, v[q].z, v[q].w);
            }
            if (kOwn) {   // one copy of this code, whatever the stage and token: it is met cold
                uint8_t* tile = smem + i % NS * p.stage_bytes + 2 * kATile + half * 2 * p.mp * kRow;
                uint8_t* atom = smem + i % NS * p.stage_bytes + 2 * kATile + 4 * p.mp * kRow + half * p.sfb_bytes;
                uint2 x[4];
                uint32_t scales = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[q] = xv[0][q];
                    uint32_t b = sv[0][q];
#pragma unroll
                    for (int u = 1; u < (kOwn ? kOwnStages : 1); ++u)
                        if (i == u) x[q] = xv[u][q], b = sv[u][q];
                    scales |= b << (8 * q);
                }
#pragma unroll 1
                for (int t = warp & 3; t < mt; t += 4) {
                    const Parts z = split4(x[0]);
                    x[0] = x[1], x[1] = x[2], x[2] = x[3];
                    *reinterpret_cast<uint32_t*>(tile + tile_at(t, lane)) = z.hi;
                    *reinterpret_cast<uint32_t*>(tile + tile_at(p.mp + t, lane)) = z.lo;
                    if ((lane & 7) == 0) {
                        atom[atom_at(t, lane >> 3)] = static_cast<uint8_t>(z.s_hi);
                        atom[atom_at(p.mp + t, lane >> 3)] = static_cast<uint8_t>(z.s_lo);
                    }
                }
                uint8_t* sfa = smem + i % NS * p.stage_bytes + 2 * kATile + p.b_bytes + half * kAtom;
                *reinterpret_cast<uint32_t*>(sfa + 16 * lane + 4 * (warp & 3)) = scales;
            }
            fence_async_proxy();   // generic writes -> the tensor core's reads
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[i % NS]);
                mbar_arrive(&code_empty[i % CS]);
            }
            return true;
        };
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) ok = spread(i);
        if (!ok) {
            s_abort = 1;
            record_status(a.status, MXFP4_ERR_TIMEOUT);
        }
    } else if (warp == 11) {
        // ---------------- packed codes
        if (lane == 0) {
            bool ok = true;
            int i = min(n, CS);
            for (; i < n; ++i) {
                if (!mbar_wait(&code_empty[i % CS], ((i / CS) & 1) ^ 1, &s_abort)) { ok = false; break; }
                load_codes(i);
            }
            if (!ok) {
                s_abort = 1;
                record_status(a.status, MXFP4_ERR_TIMEOUT);
            }
            // every slot's last copy lands before the CTA ends
            for (int w = i > CS ? i - CS : 0; w < i; ++w) mbar_wait(&code_full[w % CS], (w / CS) & 1, &s_never);
        }
    } else if (warp == 8) {
        // ---------------- prepared activations and scales
        if (!kOwn && lane == 0) {
            grid_wait();   // the prepare kernel's writes are complete
            bool ok = true;
            for (int i = 0; i < n; ++i) {
                const int s = i % NS;
                if (!mbar_wait(&empty[s], ((i / NS) & 1) ^ 1, &s_abort)) { ok = false; break; }
                uint8_t* dst = smem + s * p.stage_bytes + 2 * kATile;
                mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(p.b_bytes + 2 * kAtom));
                bulk_load(dst, ws_b + (tt * p.nk + j0 + i) * p.b_bytes, static_cast<uint32_t>(p.b_bytes), &full[s]);
                bulk_load(dst + p.b_bytes, ws_sfa + (f * p.nk + j0 + i) * (2 * kAtom), 2 * kAtom, &full[s]);
            }
            if (!ok) {
                s_abort = 1;
                record_status(a.status, MXFP4_ERR_TIMEOUT);
                // let the copies in flight land: no barrier counts them alone, so a millisecond, far
                // longer than a copy takes
                const uint64_t w0 = globaltimer_ns();
                while (globaltimer_ns() - w0 < 1000000ull) {}
            }
        }
    } else if (warp == 9) {
        // ---------------- MMA issuer (the whole warp walks the loop, one lane issues)
        bool ok = true;
        const bool lead = elect_one();
        const uint32_t idesc = idesc_mxf8(p.stacked ? 2 * p.mp : p.mp, 0);
        constexpr uint32_t kNextId = (1u << 4) | (1u << 29);
        const uint32_t tile_b = 2 * p.mp * kRow;                                  // a half's hi and lo rows
        const uint32_t lo_b = static_cast<uint32_t>(p.mp * kRow) >> 4;            // lo rows behind the hi rows
        const uint32_t sfb_at = 2 * kATile + 2 * tile_b, sfa_at = 2 * kATile + p.b_bytes;
        for (int i = 0; i < n; ++i) {
            const int s = i % NS;
            if (!__all_sync(0xFFFFFFFFu, wait_poll(&full[s], (i / NS) & 1, &s_abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(smem) + s * p.stage_bytes;
            const int steps = (k_left - 256 * i) / 32;
            if (lead) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    if (static_cast<int>(4 * h) < steps) {
                        const uint32_t set = tmem + kSfCol + 32 * (i & 1) + 16 * h;
                        const uint64_t da = sw128_desc(st + h * kATile), db = sw128_desc(st + 2 * kATile + h * tile_b);
                        tmem_cp_32x128b_x4(set, rows16_desc(st + sfa_at + h * kAtom));
                        tmem_cp_32x128b_x4(set + 4, rows16_desc(st + sfb_at + h * p.sfb_bytes));
                        if (!p.stacked) tmem_cp_32x128b_x4(set + 8, rows16_desc(st + sfb_at + h * p.sfb_bytes + kAtom));
#pragma unroll
                        for (uint32_t q = 0; q < 4; ++q) {   // 32 elements of K per MMA, scale q of the half
                            if (static_cast<int>(4 * h + q) < steps) {
                                mma_mxf8f6f4(tmem, da + 2 * q, db + 2 * q, idesc + q * kNextId, set | (q << 30),
                                             (set + 4) | (q << 30), (i | h | q) != 0 ? 1u : 0u);
                                if (!p.stacked)
                                    mma_mxf8f6f4(tmem, da + 2 * q, db + lo_b + 2 * q, idesc + q * kNextId, set | (q << 30),
                                                 (set + 8) | (q << 30), 1u);
                            }
                        }
                    }
                }
                tc_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (lead) {
            if (!ok) {
                s_abort = 1;
                record_status(a.status, MXFP4_ERR_TIMEOUT);
            }
            tc_commit(done);   // also drains every MMA issued before TMEM is released
        }
    }
    __syncwarp();

    // ---------------- the finish: each CTA of the cluster takes a share of the tokens, a thread four
    // features of every kStep-th token.  What it adds to the sums is loaded while the last MMAs run.
    constexpr int kQuads = kFeat / 4, kStep = kThreads / kQuads;
    constexpr int kBatch = SPLIT >= 3 ? 1 : 4 / SPLIT;   // tokens whose loads are in flight together
    const int c0 = rank * mt / SPLIT, c1 = (rank + 1) * mt / SPLIT;
    const int qd = tid % kQuads;
    const int64_t n0 = f * kFeat + 4 * qd;
    const bool vec = a.n_out % 4 == 0;
    const uint16_t* res = static_cast<const uint16_t*>(a.residual);
    float bz[4], bu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool in = n0 + j < a.n_out;
        bz[j] = in ? bias_at(a, n0 + j) : 0.f;
        bu[j] = kGated && in ? bias_at(a, n0 + j + a.n_out) : 0.f;
    }
    uint2 r[kBatch];
    auto load_res = [&](int c) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            r[b] = make_uint2(0u, 0u);
            if (res && c + b * kStep < c1) {
                const uint16_t* at = res + (t0 + c + b * kStep) * a.n_out + n0;
                if (vec) {
                    if (n0 < a.n_out) r[b] = *reinterpret_cast<const uint2*>(at);
                } else {
                    uint32_t half[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) half[j] = n0 + j < a.n_out ? at[j] : 0u;
                    r[b] = make_uint2(half[0] | half[1] << 16, half[2] | half[3] << 16);
                }
            }
        }
    };
    load_res(c0 + tid / kQuads);

    // ---------------- partial sums -> shared memory [token][128 rows] (the idle ring)
    const bool got = mbar_wait(done, 0, &s_never);   // suspends: a spinning warp slows the issuer
    if (!__all_sync(0xFFFFFFFFu, got)) {
        s_abort = 1;
        record_status(a.status, MXFP4_ERR_TIMEOUT);
    }
    tc_fence_after();
    __syncthreads();   // no copy into the ring is in flight: its last stage has been multiplied
    float* part = reinterpret_cast<float*>(smem);
    {
        const int q = warp & 3;
        const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16);
        float* to_row = part + 32 * q + lane;
        // 16 columns at a time; the columns behind the tile's tokens (mp = 8, or an odd half) hold
        // other rows' sums or nothing, and land behind the rows that are read
        for (int c = 16 * (warp >> 2); c < mt; c += 16 * (kThreads / 128)) {
            uint32_t v[16], w[16];
            tmem_ld_x16(base + c, v);
            if (p.stacked) tmem_ld_x16(base + p.mp + c, w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float z = __uint_as_float(v[j]);
                if (p.stacked) z += __uint_as_float(w[j]);
                to_row[(c + j) * kBM] = z;
            }
        }
    }
    __syncwarp();
    if (SPLIT > 1) cluster_sync_all(); else __syncthreads();

    {
        const uint32_t mine = smem_u32(part) + 16 * qd;
        uint16_t* y = static_cast<uint16_t*>(a.y);
        if (n0 < a.n_out) {
            for (int c = c0 + tid / kQuads; c < c1; c += kBatch * kStep) {
                float4 v[kBatch][SPLIT], w[kBatch][SPLIT];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int cc = c + b * kStep;
                    if (cc < c1) {
#pragma unroll
                        for (int q = 0; q < SPLIT; ++q) {
                            const uint32_t at = mine + cc * (kBM * 4);
                            if (SPLIT > 1) {
                                const uint32_t from = in_rank(at, q);
                                v[b][q] = ld_cluster_f32x4(from);
                                if (kGated) w[b][q] = ld_cluster_f32x4(from + 64 * 4);
                            } else {
                                const float* at_own = part + cc * kBM + 4 * qd;
                                v[b][q] = *reinterpret_cast<const float4*>(at_own);
                                if (kGated) w[b][q] = *reinterpret_cast<const float4*>(at_own + 64);
                            }
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int cc = c + b * kStep;
                    if (cc >= c1) break;
                    const int64_t m = t0 + cc, at = m * a.n_out + n0;
                    float z[4] = {v[b][0].x, v[b][0].y, v[b][0].z, v[b][0].w};
                    float u[4] = {0.f, 0.f, 0.f, 0.f};
                    if (kGated) u[0] = w[b][0].x, u[1] = w[b][0].y, u[2] = w[b][0].z, u[3] = w[b][0].w;
#pragma unroll
                    for (int q = 1; q < SPLIT; ++q) {
                        z[0] += v[b][q].x, z[1] += v[b][q].y, z[2] += v[b][q].z, z[3] += v[b][q].w;
                        if (kGated) u[0] += w[b][q].x, u[1] += w[b][q].y, u[2] += w[b][q].z, u[3] += w[b][q].w;
                    }
                    bool finite = true;
#pragma unroll
                    for (int j = 0; j < 4; ++j) finite = finite && fabsf(z[j]) < INFINITY && fabsf(u[j]) < INFINITY;
                    if (!finite) {
                        for (int j = 0; j < 4; ++j) {
                            if (n0 + j < a.n_out) {
                                z[j] = dot_direct(a, m, n0 + j);
                                if (kGated) u[j] = dot_direct(a, m, n0 + j + a.n_out);
                            }
                        }
                    }
                    float4 o = make_float4(z[0] + bz[0], z[1] + bz[1], z[2] + bz[2], z[3] + bz[3]);
                    if (kGated || a.act != MXFP4_ACT_NONE)
                        o = activate4(kGated ? static_cast<int>(MXFP4_ACT_SWIGLU) : a.act, o,
                                      make_float4(u[0] + bu[0], u[1] + bu[1], u[2] + bu[2], u[3] + bu[3]));
                    if (res) {
                        o.x += bf16_lo(r[b].x), o.y += bf16_hi(r[b].x);
                        o.z += bf16_lo(r[b].y), o.w += bf16_hi(r[b].y);
                    }
                    const uint2 out = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
                    if (vec) {
                        *reinterpret_cast<uint2*>(y + at) = out;
                    } else {
                        const uint32_t half[4] = {out.x, out.x >> 16, out.y, out.y >> 16};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (n0 + j < a.n_out) y[at + j] = static_cast<uint16_t>(half[j]);
                    }
                }
                load_res(c + kBatch * kStep);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (SPLIT > 1) cluster_sync_all();   // the partials are read: their CTAs may end
    __syncthreads();
    if (warp == 10) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// CTAs along K of a tile that prepares its own part: clusters of 4 while the GPU holds that many at once.
int own_split(const Plan& p) {
    int split = p.w_tiles <= 30 ? 4 : 2;
    while (split > p.nk) split /= 2;
    return split;
}

// The launch geometry.  Independent of the device, so that the workspace query and the call agree.
Plan make_plan(int64_t M, int64_t K, int64_t n_out, bool gated) {
    Plan p{};
    const int f = gated ? 64 : kBM;
    p.w_tiles = static_cast<int>((n_out + f - 1) / f);
    p.nk = static_cast<int>((K + 255) / 256);
    // As few token tiles as hold M (every one streams the weights), or, when those do not fill
    // the SMs and K could not be split over what is left, as many as do (400 x 2880 x 2880 21.3 -> 19.3 us,
    // 300 x 1440 x 4096 13.1 -> 12.0).
    int64_t tt = (M + kMaxMp - 1) / kMaxMp;
    if (tt > 1 && tt * p.w_tiles <= kSms && 2 * tt * p.w_tiles > kSms) tt = kSms / p.w_tiles;
    const int per = static_cast<int>((M + tt - 1) / tt);
    p.mp = per <= 8 ? 8 : (per + 15) / 16 * 16;
    p.t_tiles = static_cast<int>((M + p.mp - 1) / p.mp);
    p.stacked = 2 * p.mp <= 128;
    p.sfb_bytes = (p.stacked ? 1 : 2) * kAtom;
    p.b_bytes = 4 * p.mp * kRow + 2 * p.sfb_bytes;
    p.stage_bytes = 2 * kATile + p.b_bytes + 2 * kAtom;
    // rings: three stages where three code slots (what is in flight from memory) fit as well
    const int room = kSmemLimit - 1024 - 512;   // the base's alignment, static shared memory
    p.stages = kMaxStages;
    if (room - p.stages * p.stage_bytes < 3 * kCodeBytes) p.stages = 2;
    p.slots = (room - p.stages * p.stage_bytes) / kCodeBytes;
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    p.own = p.mp <= kOwnMp && p.t_tiles == 1 && (p.nk + own_split(p) - 1) / own_split(p) <= kOwnStages;
    return p;
}

}  // namespace

// Which engine is sooner done, by microseconds fitted to measurements.  A round of this engine's CTAs streams
// its weights again: 6 + 0.0036 K.  The other one dequantizes them once, 2.5 bytes a weight, and its
// longest pair takes 1 ns per unit of its plan's cost and stage.  One token tile is always sooner here.
// (Here and there, us: 2880 x 2880, 384 tokens 17 and 21, 512 19 and 21; 5760 x 2880 gated, 336 20 and 24,
// 384 34 and 25; 11520 x 7680, 112 37 and 82, 256 66 and 83, 384 97 and 106, 512 133 and 107.)
// K ends at 8192 because the fit does: longer ones were not measured here.  Nothing else asks for that bound (the
// prepare kernel's 32 rows of block scales fill its shared memory at K = 49000), and the other engine
// dequantizes all of W for the few tokens of such a call.
bool linear_is_few(int64_t M, int64_t K, int64_t n_out, bool gated) {
    const int64_t t = (M + kMaxMp - 1) / kMaxMp, f = gated ? 64 : kBM, w = (n_out + f - 1) / f;
    if (K > 8192) return false;
    if (t == 1) return true;
    if (t > kSms || w > (int64_t{1} << 30)) return false;
    const double here = static_cast<double>((t * w + kSms - 1) / kSms) * (6.0 + 0.0036 * static_cast<double>(K));
    const double weights = static_cast<double>(n_out) * (gated ? 2 : 1) * static_cast<double>(K);
    const double there = 8.0 + 5e-7 * weights +
                         1e-3 * static_cast<double>(linear_many_plan(M, n_out, gated, kSms).cost * ((K + 127) / 128));
    return here < there;
}

size_t linear_few_ws_bytes(int64_t M, int64_t K, int64_t n_out, bool gated) {
    const Plan p = make_plan(M, K, n_out, gated);
    if (p.own) return 0;
    return static_cast<size_t>(p.t_tiles) * p.nk * p.b_bytes + static_cast<size_t>(p.w_tiles) * p.nk * 2 * kAtom;
}

namespace {

// The product's launch with clusters of SPLIT CTAs; with `launch` false only how many such clusters
// the GPU holds at once.
template <bool kGated, int SPLIT, bool kOwn>
cudaError_t product(const CUtensorMap& tmap_codes, const LinearArgs& a, const Plan& p, const uint8_t* ws_b,
                    const uint8_t* ws_sfa, cudaStream_t stream, bool launch, int* clusters) {
    auto kern = linear_few_kernel<kGated, SPLIT, kOwn>;
    static_assert(kMaxMp * kBM * 4 + 1024 <= kSmemLimit - 512, "the partial sums fit");
    // All of the SM's shared memory, whatever the rings take: a CTA waits for its cluster while it holds
    // TMEM, so it must not share the SM with a CTA of another cluster that may wait for TMEM.
    const int smem = kSmemLimit - 512;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.w_tiles * SPLIT), static_cast<unsigned>(p.t_tiles), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(SPLIT);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // after the prepare kernel
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kOwn ? 1 : 2;
    if (launch) return cudaLaunchKernelEx(&cfg, kern, tmap_codes, a, p, ws_b, ws_sfa);
    // what a device of this kind holds does not change: asked once per kernel and tile size
    static std::atomic<int> known[kMaxMp / 8 + 1];
    std::atomic<int>& k = known[p.mp / 8];
    if ((*clusters = k.load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    if (cudaOccupancyMaxActiveClusters(clusters, kern, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();   // clear a refusal: no such cluster fits
        *clusters = 0;
    }
    k.store(*clusters, std::memory_order_relaxed);
    return cudaSuccess;
}

template <bool kGated, bool kOwn>
cudaError_t product_of(int split, const CUtensorMap& tmap_codes, const LinearArgs& a, const Plan& p, const uint8_t* ws_b,
                       const uint8_t* ws_sfa, cudaStream_t stream, bool launch, int* clusters) {
    switch (split) {
        case 1: return product<kGated, 1, kOwn>(tmap_codes, a, p, ws_b, ws_sfa, stream, launch, clusters);
        case 2: return product<kGated, 2, kOwn>(tmap_codes, a, p, ws_b, ws_sfa, stream, launch, clusters);
        case 4: return product<kGated, 4, kOwn>(tmap_codes, a, p, ws_b, ws_sfa, stream, launch, clusters);
        default: break;
    }
    if constexpr (kOwn) return cudaErrorInvalidValue;   // own_split gives at most 4
    else return product<kGated, kMaxCluster, kOwn>(tmap_codes, a, p, ws_b, ws_sfa, stream, launch, clusters);
}

// K split over the largest cluster of which the GPU holds all at once (a second round costs more than
// the split saves: 64 x 2880 x 5760 gated took 21 us with 45 clusters of 3 in two rounds, 15 with
// clusters of 2 in one).
template <bool kGated, bool kOwn>
cudaError_t launch_split(const CUtensorMap& tmap_codes, const LinearArgs& a, Plan p, const uint8_t* ws_b,
                         const uint8_t* ws_sfa, cudaStream_t stream) {
    const int64_t tiles = static_cast<int64_t>(p.w_tiles) * p.t_tiles;
    int split = kOwn ? own_split(p) : kMaxCluster;
    for (; !kOwn && split > 1; split /= 2) {
        int clusters = 0;
        if (split > p.nk || tiles * split > kSms) continue;
        cudaError_t e = product_of<kGated, kOwn>(split, tmap_codes, a, p, ws_b, ws_sfa, stream, false, &clusters);
        if (e != cudaSuccess) return e;
        if (tiles <= clusters) break;
    }
    return product_of<kGated, kOwn>(split, tmap_codes, a, p, ws_b, ws_sfa, stream, true, nullptr);
}

template <bool kGated>
cudaError_t launch_few(const LinearArgs& a, const CUtensorMap& tmap_codes, Plan p, void* ws, int sm_count,
                       cudaStream_t stream) {
    if (p.own) return launch_split<kGated, true>(tmap_codes, a, p, nullptr, nullptr, stream);
    uint8_t* ws_b = static_cast<uint8_t*>(ws);
    uint8_t* ws_sfa = ws_b + static_cast<size_t>(p.t_tiles) * p.nk * p.b_bytes;
    const int kb = static_cast<int>(a.K / 32);
    const int rows_smem = 32 * kb + 16;
    const int64_t items = a.M * ((kb + 3) / 4);
    int64_t xg = (items + kPrepareThreads / 32 - 1) / (kPrepareThreads / 32);
    if (xg > 4LL * sm_count) xg = 4LL * sm_count;
    linear_few_prepare_kernel<kGated><<<static_cast<unsigned>(4 * p.w_tiles + xg), kPrepareThreads, rows_smem, stream>>>(a, p, ws_b, ws_sfa);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_split<kGated, false>(tmap_codes, a, p, ws_b, ws_sfa, stream);
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, const CUtensorMap& tmap_codes, void* ws, int sm_count,
                              cudaStream_t stream) {
    const bool gated = a.act == MXFP4_ACT_SWIGLU;
    const Plan p = make_plan(a.M, a.K, a.n_out, gated);
    return gated ? launch_few<true>(a, tmap_codes, p, ws, sm_count, stream)
                 : launch_few<false>(a, tmap_codes, p, ws, sm_count, stream);
}

}  // namespace mx
