// few.cu -- blockwise-FP8 products for 1 to 64 tokens (sm_100a): the few-token linear
// and the two kernels of the few-token mixture-of-experts layer.
//
//   linear  y[t][n]  = sum_kb sx[t][kb] sw[n/128][kb] (sum_{k in kb} qx[t][k] qw[n][k])
//   up      g, u     = the same product of the token with an expert's gate and up rows,
//           h        = g / (1 + exp(-g)) * u, quantized per 1x128 group of h
//   down    y[t]     = sum_j weight[t][j] * (expert_j's down product of h)
//
// With so few tokens the weights are what has to be read, once, so these kernels are
// bound by HBM (by latency when the weights are small).  The product is turned over:
// 128 weight rows are the MMA's M, the tokens its N (16, 32 or 64 columns), so that one
// tcgen05.mma takes a whole 128 x 32 weight tile and TMA streams weights straight into
// shared memory without passing through registers.  An item of work is a tile of 128
// weight rows (up: 128 gate rows and the 128 up rows beside them) for the tokens of one
// expert.  The experts' CTAs walk the items; loads and products of the next item run
// while one is finished.  Where the items are fewer than the SMs, the CTAs of a cluster
// split the reduction of one item between them and join their FP32 sums through
// distributed shared memory in a fixed order.
//
//   warps 0..3  promotion: partial sums of a 128-block from TMEM (thread = weight row),
//               times weight scale x token scale, into FP32 sums in registers
//   warp 4      TMA producer: weight tiles, and the tokens' codes where memory has them
//   warps 5, 6  MMA issuers, each for one of the two TMEM buffers (one alone spends as
//               long on a block's barriers as on its products and falls behind HBM)
//   warps 7..   linear, up: quantize the tokens' 1x128 groups into shared memory (the
//               arithmetic of fp8_quant_act), one block per warp in turn; otherwise one warp
//               that loads the scales of the codes
//   the rest    experts: finish the rows of an item
//
// An expert's rows are the tokens that chose it, in their order; an item takes up to 32
// of them.  Every CTA works them out from the ids (at most 2048) before its first item:
// a 64-bit mask of tokens per expert gives each token's row by counting bits.  Columns of
// the MMA without a token hold whatever the stage held before: columns do not mix, and
// theirs are not stored.  Every wait is bounded.
//
// Measured on the device, weights from HBM (one B200, 6.5 TB/s copy rate):
//   linear  1 token 2048 x 2048 4.5 us; 7 tokens 2048 x 6144 7.0 us; 8 tokens 12288 x 2048
//           9.3 us (2.7 TB/s: 96 tiles on 148 SMs); 1 token 12288 x 12288 29.0 us (5.2 TB/s)
//   codes   61 tokens 12288 x 2048 13.7 us with the quantizer's launch (2.0 TB/s: 96 tiles on
//           148 SMs, which a cluster of 3 does not fit); 64 tokens 12288 x 12288 43.2 us (3.6
//           TB/s)
//   layer   128 experts of 2048 x 768, 8 choices: 1 token 21.5 us (start-up, join and
//           combination are most of it); 8 tokens 60 us (4.0 TB/s); 40 tokens 111 us (5.1
//           TB/s); 64 tokens 127 us (4.7 TB/s)
// The layer of many tokens is bound by HBM and by starts and ends.  At 40 tokens up's first
// product is done after 11 us (the tokens' groups wait behind the first weights), and as an
// SM takes whole items, 4.8 of them on average, up's SMs end between 59 and 77 us; down,
// which may only multiply once all have, ends at 113 to 115.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch_cache.cuh"
#include "moe.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "quant_math.cuh"
#include "tensor_map.cuh"

namespace fp8bw {

__device__ int g_few_error;  // first error code of a bounded wait in these kernels
constexpr uint64_t FEW_WAIT_NS = 1000000000ull;
constexpr uint64_t FEW_DRAIN_NS = 20000000ull;
enum : int { FERR_PRODUCER = 31, FERR_MMA_FULL = 32, FERR_MMA_TEMPTY = 33, FERR_PROMO = 34, FERR_ACT = 35, FERR_FINISH = 36 };

// FEW_CODES: the linear on codes that fp8_quant_act's kernel has made.
enum : int { FEW_LINEAR = 0, FEW_UP = 1, FEW_DOWN = 2, FEW_CODES = 3 };

constexpr int FEW_MAX_SPLIT = 8;  // CTAs of a cluster

struct FewArgs {
    const __nv_bfloat16 *x;  // [T][K] (linear, up)
    const float *sw;         // weight block scales [E][N/128][K/128]
    const int32_t *ids;      // [T][k] (up, down)
    const float *weights;    // [T][k] (down)
    __nv_bfloat16 *y;        // [T][N] (linear, codes, down)
    uint8_t *hq;             // [T*k][I] codes of h, rows by expert (up writes)
    float *hs;               // [I/128][T*k] their scales (up writes)
    const float *sx;         // [K/128][sx_rows] scales of the codes (down, codes)
    int sx_rows;
    float *part;             // [T*k][H] products of each row (down)
    int *count;              // [T][H/128] experts of the token that are done (down)
    int T, k, E;
    int N, K, KB;            // rows and columns of one expert's weight, K / 128
    int tiles_h;             // H / 128 (up clears the counters)
    uint32_t tiles_inv;      // 2^32 / tiles of an expert's weight, rounded up (at most 2^32 - 1)
    int part_lo[FEW_MAX_SPLIT + 1];  // first block of each part of the reduction
};

template <int KIND_, int NT_>
struct FewCfg {
    static constexpr int KIND = KIND_;
    static constexpr bool EXPERTS = KIND == FEW_UP || KIND == FEW_DOWN;
    static constexpr bool QUANT = KIND == FEW_LINEAR || KIND == FEW_UP;
    static constexpr int NT = NT_;                      // token columns of the MMA
    static constexpr int RT = KIND == FEW_UP ? 2 : 1;   // 128-row tiles: gate and up, or one
    static constexpr int W_BYTES = RT * 128 * 128;
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    // CTAs per SM: one with a deep ring where many items stream through it; two where a
    // few items' latency counts, so that one's start runs under the other's loads (and
    // down's under up's).
    static constexpr int BLOCKS = EXPERTS && NT > 16 ? 1 : 2;
    static constexpr int ACT_WARP0 = 7;
    static constexpr int ACT_WARPS = KIND == FEW_LINEAR ? 4 : KIND == FEW_UP ? 2 : 1;
    static constexpr int ROW_PAIRS = KIND == FEW_UP && BLOCKS == 2 ? 2 : 4;  // quantized at a time
    static constexpr int FIN_WARP0 = ACT_WARP0 + ACT_WARPS;
    // Up has three: 12 warps leave its promotion warps the registers for their sums.  Down's
    // rows wait for memory three times over, about as long as an item's products take.
    static constexpr int FIN_WARPS = KIND == FEW_UP ? 3 : KIND != FEW_DOWN ? 0 : BLOCKS == 1 ? 8 : 4;
    static constexpr int RBUF = KIND == FEW_DOWN ? 2 : 1;  // items that may wait to be finished
    static constexpr int THREADS = (FIN_WARP0 + FIN_WARPS) * 32;
    static constexpr int NBUF = 2;
    static constexpr int TMEM_COLS = NBUF * RT * NT;    // 32 .. 128, a power of two
    // finished sums of the items, [RBUF][NT][128]; before the first, scratch of the plan
    static constexpr int RED_BYTES = EXPERTS ? RBUF * NT * 128 * 4 : 0;
    static constexpr int MAX_PAIRS = !EXPERTS ? 0 : NT == 16 ? 16 * 32 : 64 * 32;
    static constexpr int MAX_UNITS = !EXPERTS ? 0 : (NT == 16 ? MAX_PAIRS : 1024) + MAX_PAIRS / NT;
    static constexpr int FIXED = RED_BYTES + (EXPERTS ? 1024 * 10 : 0) + MAX_UNITS * 4 + MAX_PAIRS + 1536;
    static constexpr int STAGES = (226 / BLOCKS * 1024 - FIXED) / (STAGE_BYTES + NT * 4);
    static constexpr int RED_OFF = STAGES * STAGE_BYTES;
    static constexpr int XS_OFF = RED_OFF + RED_BYTES;          // [STAGES][NT] token scales
    static constexpr int MASK_OFF = XS_OFF + STAGES * NT * 4;   // [1024][2] unsigned
    static constexpr int BASE_OFF = MASK_OFF + (EXPERTS ? 1024 * 8 : 0);  // [1024] 16-bit
    static constexpr int UNIT_OFF = BASE_OFF + (EXPERTS ? 1024 * 2 : 0);  // [MAX_UNITS] unsigned
    static constexpr int TOKEN_OFF = UNIT_OFF + MAX_UNITS * 4;  // [MAX_PAIRS] 8-bit
    static constexpr int BAR_OFF = TOKEN_OFF + MAX_PAIRS;
    static constexpr int SMEM = 1024 + BAR_OFF + (2 * STAGES + 2 * NBUF + 2 * RBUF) * 8 + 16;
    static_assert(BAR_OFF % 8 == 0, "barriers are 8-byte words");
    static_assert(RT * NT * 128 * 4 <= STAGES * STAGE_BYTES, "a cluster's parts take the stages");
    static_assert(MAX_PAIRS * 2 <= RED_BYTES, "the plan's scratch");
    // 228 KB per SM, 1 KB of it reserved per CTA
    static_assert((SMEM + 1024 + 64) * BLOCKS <= 228 * 1024, "shared memory of an SM");
};

// Some of one expert's rows, packed into a word: expert, first row (among all experts'),
// how many.
struct FewUnit {
    int expert, base, rows;
    __device__ __forceinline__ static uint32_t pack(int expert, int base, int rows)
    {
        return uint32_t(expert) << 20 | uint32_t(base) << 8 | uint32_t(rows);
    }
    __device__ __forceinline__ static FewUnit of(uint32_t w)
    {
        return {int(w >> 20), int(w >> 8 & 0xFFFu), int(w & 0xFFu)};
    }
};

// The experts' rows, in shared memory.
struct FewPlan {
    uint32_t *mask;   // [E][2] the tokens that chose each expert
    uint16_t *base;   // [E] its first row
    uint32_t *units;  // the units of all experts
    uint8_t *token;   // of each row

    // How many of expert e's tokens come before t.
    __device__ __forceinline__ int before(int e, int t) const
    {
        const uint32_t low = (1u << (t & 31)) - 1u;
        return t < 32 ? __popc(mask[2 * e] & low) : __popc(mask[2 * e]) + __popc(mask[2 * e + 1] & low);
    }
    __device__ __forceinline__ int row(int e, int t) const { return base[e] + before(e, t); }

    // make_units from the ids of at most 32 pairs, a lane each (-1: none), whatever E: one
    // step in the place of one per 32 experts.  The experts stand in the order in which the
    // pairs name them; up and down make the same order, which nothing else depends on.
    template <int NT> __device__ __forceinline__ int make_units_of(int id, int E, int lane) const
    {
        const uint32_t live = __ballot_sync(0xffffffffu, id >= 0);
        const uint32_t same = same_key(uint32_t(id), 32 - __clz(E - 1)) & live;
        const bool first = id >= 0 && __ffs(same) - 1 == lane;
        const int c = first ? __popc(mask[2 * id]) + __popc(mask[2 * id + 1]) : 0;
        const int u = (c + NT - 1) / NT;
        int sum = u << 16 | c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= o ? up : 0;
        }
        const int row0 = (sum & 0xFFFF) - c, unit = (sum >> 16) - u;
        if (first)
            base[id] = uint16_t(row0);
        for (int i = 0; i < u; ++i)
            units[unit + i] = FewUnit::pack(id, row0 + i * NT, min(NT, c - i * NT));
        return __shfl_sync(0xffffffffu, sum, 31) >> 16;
    }

    // Masks -> first rows and units of at most NT rows.  One warp; returns how many units.
    template <int NT> __device__ __forceinline__ int make_units(int E, int lane) const
    {
        int row0 = 0, unit0 = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? __popc(mask[2 * e]) + __popc(mask[2 * e + 1]) : 0;
            const int u = (c + NT - 1) / NT;
            int sum = u << 16 | c;  // both sums at once: at most 2048 rows and 1088 units
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                sum += lane >= o ? up : 0;
            }
            const int first = row0 + (sum & 0xFFFF) - c, unit = unit0 + (sum >> 16) - u;
            if (e < E)
                base[e] = uint16_t(first);
            for (int i = 0; i < u; ++i)
                units[unit + i] = FewUnit::pack(e, first + i * NT, min(NT, c - i * NT));
            const int all = __shfl_sync(0xffffffffu, sum, 31);
            row0 += all & 0xFFFF;
            unit0 += all >> 16;
        }
        return unit0;
    }
};

__device__ __forceinline__ uint2 bf16x4(float4 v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

__device__ __forceinline__ float swiglu(float g, float u)
{
    return g / (1.0f + expf(-g)) * u;
}

// Lane j: choice j of token t, -1 where it is left out.
__device__ __forceinline__ int few_choice(const FewArgs &a, int t, int lane)
{
    const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    return id >= 0 && id < a.E ? id : -1;
}

// One row of an item, finished by one warp: lane l has columns 4 l .. 4 l + 3 of its tile
// (g, u: of the gate and up rows; otherwise v).
__device__ __forceinline__ void few_store(const FewArgs &a, int r, int tile, int lane, float4 v)
{
    *reinterpret_cast<uint2 *>(a.y + size_t(r) * a.N + tile * 128 + 4 * lane) = bf16x4(v);
}

__device__ __forceinline__ void few_store_h(const FewArgs &a, int row, int tile, int lane, float4 h)
{
    // the largest magnitude by its bits, whose order is that of the numbers with NaN above
    // them all: a NaN reaches the scale (fmaxf would drop it), as in the quantizers
    const uint32_t most = max(max(__float_as_uint(fabsf(h.x)), __float_as_uint(fabsf(h.y))),
                              max(__float_as_uint(fabsf(h.z)), __float_as_uint(fabsf(h.w))));
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
    // h is kept in FP32 up to its one rounding onto E4M3
    const float sc = __fdiv_rn(amax, 448.0f);
    uint32_t codes = 0u;
    if (sc != 0.0f)
        codes = cvt_e4m3x2(__fdiv_rn(h.x, sc), __fdiv_rn(h.y, sc)) |
                (cvt_e4m3x2(__fdiv_rn(h.z, sc), __fdiv_rn(h.w, sc)) << 16);
    *reinterpret_cast<uint32_t *>(a.hq + size_t(row) * (a.N / 2) + tile * 128 + 4 * lane) = codes;
    if (lane == 0)
        a.hs[size_t(tile) * (a.T * a.k) + row] = sc;
}

// The row's product goes to memory; the warp that brings a token's last one adds them
// all, in the order of the choices.
__device__ __forceinline__ void few_combine(const FewArgs &a, const FewPlan &p, int row, int tile,
                                            int lane, float4 v)
{
    const int t = p.token[row];
    const size_t col = size_t(tile) * 128 + 4 * lane;
    *reinterpret_cast<float4 *>(a.part + size_t(row) * a.N + col) = v;
    const int id = few_choice(a, t, lane);
    const float weight = lane < a.k ? a.weights[t * a.k + lane] : 0.0f;
    // choices that name the same expert share its row
    const uint32_t live = __ballot_sync(0xffffffffu, id >= 0);
    const uint32_t same = same_key(uint32_t(id), 32 - __clz(a.E - 1)) & live;
    const uint32_t rows = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
    __threadfence();
    __syncwarp();
    int done = 0;
    if (lane == 0)
        done = atomicAdd(&a.count[t * (a.N / 128) + tile], 1) + 1;
    done = __shfl_sync(0xffffffffu, done, 0);
    if (done != __popc(rows))
        return;
    __threadfence();
    const int at = id >= 0 ? p.row(id, t) : 0;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const float w = __shfl_sync(0xffffffffu, weight, j);
        const int r = __shfl_sync(0xffffffffu, at, j);
        if (!((live >> j) & 1u))
            continue;
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(a.part + size_t(r) * a.N + col));
        y.x = fmaf(w, q.x, y.x);
        y.y = fmaf(w, q.y, y.y);
        y.z = fmaf(w, q.z, y.z);
        y.w = fmaf(w, q.w, y.w);
    }
    few_store(a, t, tile, lane, y);
}

// Quantizes up to 2 P rows of one 128-block: half-warp h takes rows r0 + 2 q + h, lane
// `sub` of it 8 neighbouring values (v[q]).  The P chains of maximum, scale and division
// run side by side.
template <int P>
__device__ __forceinline__ void few_quant(const uint4 (&v)[P], int r0, int rows, int lane, uint8_t *sx,
                                          float *xs)
{
    const int sub = lane & 15;
    uint32_t m2[P];
#pragma unroll
    for (int q = 0; q < P; ++q)
        m2[q] = __vmaxu2(absmax2(v[q].x, v[q].y), absmax2(v[q].z, v[q].w));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
        for (int q = 0; q < P; ++q)
            m2[q] = __vmaxu2(m2[q], __shfl_xor_sync(0xffffffffu, m2[q], o));
    float sc[P];
    bool fast = true;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        sc[q] = scale_of_amax(halves_max_to_float(m2[q]));
        fast = fast && (m2[q] == 0u || (sc[q] >= 0x1p-90f && sc[q] <= 0x1p90f));
    }
    uint2 c[P];
    if (__all_sync(0xffffffffu, fast)) {
#pragma unroll
        for (int q = 0; q < P; ++q)
            c[q] = quant8_fast(v[q], __frcp_rn(m2[q] ? sc[q] : 1.0f), sc[q]);
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q)
            c[q] = quant8_ieee(v[q], sc[q]);
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int r = r0 + 2 * q + (lane >> 4);
        if (r < rows) {
            *reinterpret_cast<uint2 *>(sx + r * 128 + (((sub >> 1) ^ (r & 7)) << 4) + (sub & 1) * 8) =
                m2[q] ? c[q] : make_uint2(0u, 0u);  // an all-zero group has codes 0
            if (sub == 0)
                xs[r] = sc[q];
        }
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::BLOCKS)
few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH,
           const FewArgs a)
{
    constexpr int KIND = Cfg::KIND, NT = Cfg::NT, RT = Cfg::RT, STAGES = Cfg::STAGES;
    constexpr int NBUF = Cfg::NBUF, WARPS = Cfg::THREADS / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(smem + Cfg::RED_OFF);
    float *xs = reinterpret_cast<float *>(smem + Cfg::XS_OFF);
    const FewPlan plan = {reinterpret_cast<uint32_t *>(smem + Cfg::MASK_OFF),
                          reinterpret_cast<uint16_t *>(smem + Cfg::BASE_OFF),
                          reinterpret_cast<uint32_t *>(smem + Cfg::UNIT_OFF), smem + Cfg::TOKEN_OFF};
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + NBUF;
    uint64_t *rfull = tempty + NBUF, *rempty = rfull + Cfg::RBUF;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rempty + Cfg::RBUF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    __shared__ int unit_count;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = int(cluster_ctarank()), split = int(cluster_nctarank());
    const int first = int(cluster_id_x()), step = int(cluster_count_x());
    int16_t *id = reinterpret_cast<int16_t *>(red);  // scratch of the plan: the pairs' ids

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);   // the producer's bytes, and the codes or scales
            mbar_init(&empty[s], 4);  // the promotion warps, when the MMA is done
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 4);
        }
        for (int b = 0; b < Cfg::RBUF; ++b) {
            mbar_init(&rfull[b], 4);
            mbar_init(&rempty[b], Cfg::EXPERTS ? Cfg::FIN_WARPS : 1);
        }
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmW);
    }
    if (Cfg::EXPERTS)
        for (int i = tid; i < 2 * a.E; i += Cfg::THREADS)
            plan.mask[i] = 0;
    if (warp == 5) {
        tmem_alloc<1>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // The tensor memory is held before a dependent kernel may start: one that started
    // first and took it would wait for this one, which would wait for it.
    if (Cfg::QUANT) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // down, codes: the kernel before this one (up; the quantizer) waited for its own
    // predecessor before it let this one start, so the ids and the weights are complete
    // and only what that kernel writes has to be waited for
    if (Cfg::QUANT) {
        // The tokens on their way to L2 before the weights take the memory's queues, a
        // line for each thread of the grid (what that does not reach is loaded later).
        const int64_t line = int64_t(blockIdx.x) * Cfg::THREADS + tid;
        if (line < int64_t(a.T) * a.K / 64)
            prefetch_l2(a.x + line * 64);
    }
    if (KIND == FEW_UP)
        for (int i = int(blockIdx.x) * Cfg::THREADS + tid; i < a.T * a.tiles_h;
             i += int(gridDim.x) * Cfg::THREADS)
            a.count[i] = 0;
    const int n_tiles = a.N / 128, tiles = n_tiles / RT;
    int items = tiles;
    if (Cfg::EXPERTS) {
        for (int i = tid; i < a.T * a.k; i += Cfg::THREADS) {
            const int v = a.ids[i], t = i / a.k;
            const bool ok = v >= 0 && v < a.E;
            id[i] = int16_t(ok ? v : -1);
            if (ok)
                atomicOr(&plan.mask[2 * v + (t >> 5)], 1u << (t & 31));
        }
        __syncthreads();
        if (warp == 4) {
            const int pairs = a.T * a.k;
            const int n = pairs <= 32
                              ? plan.make_units_of<NT>(lane < pairs ? int(id[lane]) : -1, a.E, lane)
                              : plan.make_units<NT>(a.E, lane);
            if (lane == 0)
                unit_count = n;
        }
        __syncthreads();
        items *= unit_count;
    }
    // This CTA's items are first, first + step, ...; its part of their reduction is the
    // blocks lo .. lo + nkb - 1.  (No divisions here: nothing is loaded before this is done.)
    const int lo = a.part_lo[rank], nkb = a.part_lo[rank + 1] - lo;
    // A place in that walk: an item, and the block within its part.
    struct Walk {
        int item, i, tile;
        FewUnit u;
    };
    const auto enter = [&](Walk &w, int item) {
        w.item = item;
        w.u = {0, 0, a.T};
        w.tile = item;
        if (Cfg::EXPERTS && item < items) {
            // item / tiles by its inverse, which is off by one at most
            int unit = int(__umulhi(uint32_t(item), a.tiles_inv)), tile = item - unit * tiles;
            if (tile < 0) {
                --unit;
                tile += tiles;
            } else if (tile >= tiles) {
                ++unit;
                tile -= tiles;
            }
            w.u = FewUnit::of(plan.units[unit]);
            w.tile = tile;
        }
    };
    const auto start = [&](int i) {
        Walk w;
        enter(w, first);
        w.i = i;
        return w;
    };
    const auto advance = [&](Walk &w, int by) {
        w.i += by;
        while (w.i >= nkb) {
            w.i -= nkb;
            enter(w, w.item + step);
        }
    };
    // MMA columns in use: whole groups of 16
    const auto columns = [](int rows) { return NT <= 16 ? 16 : (rows + 15) / 16 * 16; };
    // Weights are read once: they must not push out of L2 what every item needs (codes,
    // scales, the kernel's own code, which then comes from HBM behind them).
    const uint64_t once = l2_evict_first();
    const auto load_weights = [&](const Walk &w, int s) {
        const int row = w.u.expert * a.N + w.tile * 128;
        uint8_t *dst = smem + s * Cfg::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[s], Cfg::W_BYTES + (Cfg::QUANT ? 0 : Cfg::X_BYTES));
        tma_load_2d_hint(dst, &tmW, &full[s], (lo + w.i) * 128, row, once);
        if (KIND == FEW_UP)
            tma_load_2d_hint(dst + 128 * 128, &tmW, &full[s], (lo + w.i) * 128, row + a.N / 2, once);
    };
    // weights do not wait for the order of the rows, nor for the kernel before
    int early = 0;
    if (warp == 4 && lane == 0)
        for (Walk w = start(0); early < STAGES && w.item < items; ++early, advance(w, 1))
            load_weights(w, early);
    if (Cfg::EXPERTS) {
        for (int i = tid; i < a.T * a.k; i += Cfg::THREADS)
            if (id[i] >= 0)
                plan.token[plan.row(id[i], i / a.k)] = uint8_t(i / a.k);
        __syncthreads();
    }

    if (warp < 4) {
        // ------------------------------------------------------------- promotion
        Walk at, to;
        enter(at, first);
        const float *sw[RT];  // weight scales, loaded a block ahead, across items too
        float next[RT];
        const auto scales_of = [&](const Walk &w) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
                sw[r] = a.sw + (size_t(w.u.expert) * n_tiles + w.tile + r * tiles) * a.KB + lo;
        };
        if (first < items) {
            scales_of(at);
#pragma unroll
            for (int r = 0; r < RT; ++r)
                next[r] = __ldg(sw[r]);
        }
        bool ok = true;
        for (int n = 0, m = 0; at.item < items && ok; at = to, ++m) {
            const FewUnit u = at.u;
            const int cols = columns(u.rows);
            enter(to, at.item + step);
            float2 acc[RT][NT / 2];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < NT / 2; ++c)
                    acc[r][c] = make_float2(0.0f, 0.0f);
            for (int i = 0; i < nkb; ++i, ++n) {
                const int s = n % STAGES, b = n % NBUF;
                float2 cur[RT];
                const bool more = i + 1 < nkb;
                const bool next_item = !more && to.item < items;
                if (next_item)
                    scales_of(to);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    cur[r] = make_float2(next[r], next[r]);
                    if (more || next_item)
                        next[r] = __ldg(sw[r] + (more ? i + 1 : 0));
                }
                // the stage's full barrier cannot run ahead: it waits for this warp below
                ok = mbar_wait_bounded(&full[s], uint32_t(n / STAGES) & 1u, abort_flag, &g_few_error,
                                       FERR_PROMO, FEW_WAIT_NS) &&
                     mbar_wait_bounded(&tfull[b], uint32_t(n / NBUF) & 1u, abort_flag, &g_few_error,
                                       FERR_PROMO, FEW_WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t taddr =
                    tmem_base + (uint32_t(warp * 32) << 16) + uint32_t(b * RT * NT);
                const float4 *xs4 = reinterpret_cast<const float4 *>(xs + s * NT);
                // 16 columns of one tile at a time: the sums already take RT x NT registers
#pragma unroll
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    if (c0 >= cols)
                        break;
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(taddr + uint32_t(r * NT + c0), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 x4 = xs4[(c0 + c) / 4];
                            const float2 xc[2] = {make_float2(x4.x, x4.y), make_float2(x4.z, x4.w)};
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float2 &o = acc[r][(c0 + c) / 2 + q];
                                o = __ffma2_rn(make_float2(__uint_as_float(v[c + 2 * q]),
                                                           __uint_as_float(v[c + 2 * q + 1])),
                                               __fmul2_rn(cur[r], xc[q]), o);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&tempty[b]);
                    mbar_arrive(&empty[s]);
                }
            }
            if (!Cfg::EXPERTS || split > 1) {
                // The only item: every product of this CTA is done (the last buffer was
                // full), so the stages are free to take its parts, [RT][NT][128].
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < NT; c += 2) {
                        if (c < u.rows)
                            part[(r * NT + c) * 128 + tid] = acc[r][c / 2].x;
                        if (c + 1 < u.rows)
                            part[(r * NT + c + 1) * 128 + tid] = acc[r][c / 2].y;
                    }
                continue;
            }
            const int rb = m % Cfg::RBUF;
            float *sums = red + rb * NT * 128;
            ok = ok && __all_sync(0xffffffffu,
                                  mbar_wait_bounded(&rempty[rb], (uint32_t(m / Cfg::RBUF) & 1u) ^ 1u,
                                                    abort_flag, &g_few_error, FERR_PROMO,
                                                    FEW_WAIT_NS));
            if (!ok)
                break;
#pragma unroll
            for (int c = 0; c < NT; c += 2) {
                float2 v = acc[0][c / 2];
                if (c < u.rows) {
                    if (KIND == FEW_UP)
                        v = make_float2(swiglu(v.x, acc[RT - 1][c / 2].x),
                                        swiglu(v.y, acc[RT - 1][c / 2].y));
                    sums[c * 128 + tid] = v.x;
                }
                if (c + 1 < u.rows)
                    sums[(c + 1) * 128 + tid] = v.y;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&rfull[rb]);
        }
    } else if (warp == 4) {
        // -------------------------------------------------------------- producer
        if (lane == 0 && first < items) {
            if (!Cfg::QUANT) {
                pdl_wait();
                pdl_launch_dependents();
            }
            Walk w = start(0);
            for (int n = 0; w.item < items; ++n, advance(w, 1)) {
                const int s = n % STAGES;
                if (n >= early) {
                    if (!mbar_wait_bounded(&empty[s], (uint32_t(n / STAGES) & 1u) ^ 1u, abort_flag,
                                           &g_few_error, FERR_PRODUCER, FEW_WAIT_NS))
                        break;
                    load_weights(w, s);
                }
                if (!Cfg::QUANT)
                    tma_load_2d(smem + s * Cfg::STAGE_BYTES + Cfg::W_BYTES, &tmH, &full[s],
                                (lo + w.i) * 128, w.u.base);
            }
        }
    } else if (warp < Cfg::ACT_WARP0) {
        // ------------------------------------------------------------------- MMA
        if (lane == 0) {
            static_assert(NBUF == 2, "one MMA warp per buffer");
            const int b = warp - 5;
            Walk w = start(0);
            advance(w, b);
            for (int n = b; w.item < items; n += NBUF, advance(w, NBUF)) {
                const int s = n % STAGES;
                const uint32_t idesc = make_idesc_e4m3(128, columns(w.u.rows), 0);
                if (!mbar_spin_bounded(&full[s], uint32_t(n / STAGES) & 1u, abort_flag, &g_few_error,
                                       FERR_MMA_FULL, FEW_WAIT_NS) ||
                    !mbar_spin_bounded(&tempty[b], (uint32_t(n / NBUF) & 1u) ^ 1u, abort_flag,
                                       &g_few_error, FERR_MMA_TEMPTY, FEW_WAIT_NS))
                    break;
                tc_fence_after();
                const uint32_t w_addr = smem_u32(smem + s * Cfg::STAGE_BYTES);
                const uint32_t x_addr = w_addr + Cfg::W_BYTES;
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8f6f4<1>(tmem_base + uint32_t((b * RT + r) * NT),
                                      make_smem_desc_sw128(w_addr + r * 128 * 128 + k * 32, 16, 1024),
                                      make_smem_desc_sw128(x_addr + k * 32, 16, 1024), idesc,
                                      k > 0 ? 1u : 0u);
                mma_commit(&tfull[b]);
            }
        }
    } else if (Cfg::EXPERTS && warp >= Cfg::FIN_WARP0) {
        // --------------------------------------------------------- finish the rows
        // Rows go to the warps in turn, on from the item before: most items have fewer rows
        // than there are warps, and a row of down takes about as long as an item's products.
        constexpr int FIN = Cfg::FIN_WARPS > 0 ? Cfg::FIN_WARPS : 1;
        Walk at;
        for (int item = first, m = 0, turn = 0; item < items && split == 1; item += step, ++m) {
            enter(at, item);
            const int rb = m % Cfg::RBUF, rows = at.u.rows;
            const bool ok = mbar_wait_bounded(&rfull[rb], uint32_t(m / Cfg::RBUF) & 1u, abort_flag,
                                              &g_few_error, FERR_FINISH, FEW_WAIT_NS);
            if (!__all_sync(0xffffffffu, ok))
                break;
            int r = warp - Cfg::FIN_WARP0 - turn;
            r += r < 0 ? FIN : 0;
            turn = (turn + rows) % FIN;
            const float *sums = red + rb * NT * 128 + 4 * lane;
            if (KIND == FEW_DOWN) {
                // all of this warp's sums first: the buffer is free before the rows are done
                constexpr int MINE = (NT + FIN - 1) / FIN;
                float4 v[MINE];
#pragma unroll
                for (int i = 0; i < MINE; ++i)
                    if (r + i * FIN < rows)
                        v[i] = *reinterpret_cast<const float4 *>(sums + (r + i * FIN) * 128);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&rempty[rb]);
#pragma unroll
                for (int i = 0; i < MINE; ++i)
                    if (r + i * FIN < rows)
                        few_combine(a, plan, at.u.base + r + i * FIN, at.tile, lane, v[i]);
            } else {
                for (; r < rows; r += FIN)
                    few_store_h(a, at.u.base + r, at.tile, lane,
                                *reinterpret_cast<const float4 *>(sums + r * 128));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&rempty[rb]);
            }
        }
    } else if (Cfg::QUANT) {
        // -------------------------------------------- quantize the tokens' groups
        // One block per warp in turn, a few row pairs at a time, the next ones' values under
        // way meanwhile.
        constexpr int P = Cfg::ROW_PAIRS;
        const uint4 *x4 = reinterpret_cast<const uint4 *>(a.x) + lo * 16 + (lane & 15);
        const auto fetch = [&](const Walk &w, int r0, uint4 (&v)[P]) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int r = r0 + 2 * q + (lane >> 4);
                v[q] = make_uint4(0u, 0u, 0u, 0u);
                if (w.item < items && r < w.u.rows) {
                    const int t = KIND == FEW_UP ? int(plan.token[w.u.base + r]) : r;
                    v[q] = __ldg(x4 + (t * (a.K / 8) + w.i * 16));
                }
            }
        };
        uint4 v[P], ahead[P];
        Walk w = start(0), next;
        advance(w, warp - Cfg::ACT_WARP0);
        fetch(w, 0, v);
        for (int n = warp - Cfg::ACT_WARP0; w.item < items; n += Cfg::ACT_WARPS, w = next) {
            const int s = n % STAGES, rows = w.u.rows;
            next = w;
            advance(next, Cfg::ACT_WARPS);
            const bool ok = mbar_wait_bounded(&empty[s], (uint32_t(n / STAGES) & 1u) ^ 1u, abort_flag,
                                              &g_few_error, FERR_ACT, FEW_WAIT_NS);
            if (!__all_sync(0xffffffffu, ok))
                break;
            uint8_t *sx = smem + s * Cfg::STAGE_BYTES + Cfg::W_BYTES;
            for (int r0 = 0; r0 < rows; r0 += 2 * P) {
                const bool more = r0 + 2 * P < rows;
                fetch(more ? w : next, more ? r0 + 2 * P : 0, ahead);
                if (r0 + 2 < rows) {
                    few_quant<P>(v, r0, rows, lane, sx, xs + s * NT);
                } else {
                    const uint4 one[1] = {v[0]};
                    few_quant<1>(one, r0, rows, lane, sx, xs + s * NT);
                }
#pragma unroll
                for (int q = 0; q < P; ++q)
                    v[q] = ahead[q];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[s]);
        }
    } else {
        // --------------------------------------------------- scales of the codes
        // A few blocks at a time, the next ones' under way meanwhile: one after the other,
        // each block would wait for memory anew (61 tokens, 12288 x 2048: 14.9 us so, 13.8 by
        // four; 64 tokens, 12288 x 12288: 46.6 and 42.8).  Down of up to 16 tokens has the
        // registers for one ahead.
        constexpr int G = Cfg::EXPERTS && Cfg::BLOCKS == 2 ? 1 : 4, PER = (NT + 31) / 32;
        // loads those of the G blocks from `from` on, and returns the place behind them
        const auto fetch = [&](Walk from, float (&v)[G][PER]) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    if (from.item < items && lane + 32 * q < from.u.rows)
                        v[g][q] = a.sx[size_t(lo + from.i) * a.sx_rows + from.u.base + lane + 32 * q];
                if (from.item < items)
                    advance(from, 1);
            }
            return from;
        };
        float v[G][PER], ahead[G][PER];
        Walk w = start(0);
        pdl_wait();
        Walk next = fetch(w, v);
        bool ok = true;
        for (int n = 0; w.item < items && ok;) {
            next = fetch(next, ahead);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (w.item >= items)
                    break;
                const int s = n % STAGES;
                ok = mbar_wait_bounded(&empty[s], (uint32_t(n / STAGES) & 1u) ^ 1u, abort_flag,
                                       &g_few_error, FERR_ACT, FEW_WAIT_NS);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    if (lane + 32 * q < w.u.rows)
                        xs[s * NT + lane + 32 * q] = v[g][q];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[s]);
                advance(w, 1);
                ++n;
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    v[g][q] = ahead[g][q];
        }
    }
    if (!Cfg::QUANT)
        pdl_wait();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // give copies and MMAs still in flight time to land before the memory is released
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < FEW_DRAIN_NS) {
        }
    }
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, Cfg::TMEM_COLS);
    }
    if (!Cfg::EXPERTS || split > 1) {
        // ---------------------------------------------------- join the cluster's parts
        if (split > 1)
            cluster_sync();
        if (first < items) {
            Walk w;
            enter(w, first);
            const FewUnit u = w.u;
            const int tile = w.tile;
            const uint32_t part0 = smem_u32(smem);
            for (int r = rank + split * warp; r < u.rows; r += split * WARPS) {
                float4 sum[RT];
#pragma unroll
                for (int q = 0; q < RT; ++q) {
                    const uint32_t at = part0 + uint32_t(((q * NT + r) * 128 + 4 * lane) * 4);
                    float4 v[FEW_MAX_SPLIT];
#pragma unroll
                    for (int p = 0; p < FEW_MAX_SPLIT; ++p)
                        v[p] = p < split ? ld_cluster_v4(mapa_shared(at, uint32_t(p)))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                    sum[q] = v[0];
#pragma unroll
                    for (int p = 1; p < FEW_MAX_SPLIT; ++p) {
                        sum[q].x += v[p].x;
                        sum[q].y += v[p].y;
                        sum[q].z += v[p].z;
                        sum[q].w += v[p].w;
                    }
                }
                const float4 g = sum[0], up = sum[RT - 1];
                if (KIND == FEW_UP)
                    few_store_h(a, u.base + r, tile, lane,
                                make_float4(swiglu(g.x, up.x), swiglu(g.y, up.y), swiglu(g.z, up.z),
                                            swiglu(g.w, up.w)));
                else if (KIND == FEW_DOWN)
                    few_combine(a, plan, u.base + r, tile, lane, g);
                else
                    few_store(a, r, tile, lane, g);
            }
        }
        if (split > 1)
            cluster_sync();  // no peer reads this CTA's parts any more
    }
    if (KIND == FEW_DOWN)
        // tokens that chose no expert: one warp for each of their tiles
        for (int i = int(blockIdx.x) * WARPS + warp; i < a.T * tiles; i += int(gridDim.x) * WARPS)
            if (!__any_sync(0xffffffffu, few_choice(a, i / tiles, lane) >= 0))
                few_store(a, i / tiles, i % tiles, lane, make_float4(0.f, 0.f, 0.f, 0.f));
}

// ------------------------------------------------------------------- host side

// Whether the linear quantizes its tokens itself.  Every tile's CTAs quantize them anew;
// beyond some tokens that takes longer than their weights take to arrive, and the codes
// come from the quantizer's kernel instead, a launch more, whose time the next one's start
// hides.  Measured (itself / codes): 8 tokens 5.0 / 6.1 us at 2048 x 2048 and 28.9 / 29.9 at
// 12288 x 12288; 16 tokens 5.6 / 5.7 (1024 x 1024), 6.3 / 6.1 (2048 x 2048), 7.1 / 6.9 (4096 x
// 2048), 9.3 / 9.4 (4096 x 4096), 11.6 / 10.3 (12288 x 2048), 13.0 / 11.2 (2048 x 12288), 12.4
// / 11.7 (8192 x 4096) and 39.2 / 30.5 (12288 x 12288); 9 tokens within 0.3 us at all of these
// but 4096 x 4096 (8.3 / 9.1) and up to 1024 x 1024 (4.9 / 5.5); 32 tokens 9.6 / 7.2 at 2048 x
// 2048.
constexpr int FEW_QUANT_TOKENS = 8;        // at any size
constexpr int FEW_QUANT_TOKENS_SMALL = 16; // of a weight of at most this many elements
constexpr int64_t FEW_QUANT_SMALL = int64_t(1) << 24;

// CTAs per item: the split of the reduction that leaves an SM the least time, in blocks of
// a CTA alone: two CTAs on an SM take 0.7 of their blocks' sum (each hides the other's
// start and end), a join counts as two blocks, and each CTA has two blocks at least.
// (Measured by split, 1 .. 8: up of one token and 8 experts, 48 items of 16 blocks: 29.9 /
// 24.3 / 22.9 / 22.0 / 22.4 / 28.7 us for the layer; 7 tokens, 2048 x 6144, 16 items of 48
// blocks, by 2 .. 6 and 8: 11.5 / 9.0 / 7.9 / 7.3 / 6.8 / 6.6 us.)  All clusters have to be
// resident at once (fit[s] of them are): a second round of them costs more than any
// split gains (61 tokens, 12288 x 2048, 96 items of 16 blocks: 14.5 us split by 2, 19.8 us
// by 3, of which fewer fit).
static int few_split(int64_t items, int64_t KB, int64_t sms, const int (&fit)[FEW_MAX_SPLIT + 1])
{
    const auto cost = [&](int s) {
        const int64_t ctas = (items * s + sms - 1) / sms;
        return double(ctas * ((KB + s - 1) / s)) * (ctas > 1 ? 0.7 : 1.0) + (s > 1 ? 2.0 : 0.0);
    };
    int best = 1;
    for (int s = 2; s <= FEW_MAX_SPLIT && KB >= 2 * s; ++s)
        if (items <= fit[s] && cost(s) < cost(best))
            best = s;
    return best;
}

template <class Cfg>
static cudaError_t run_few(const uint8_t *w, int64_t w_rows, const uint8_t *codes, FewArgs a,
                           cudaStream_t stream, int num_sms)
{
    auto kern = few_kernel<Cfg>;
    static LaunchCache cache[FEW_MAX_SPLIT + 1];  // clusters of each size that fit the GPU
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (cache[FEW_MAX_SPLIT].get(dev) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
        if (e != cudaSuccess)
            return e;
        for (int s = 1; s <= FEW_MAX_SPLIT; ++s) {
            cudaLaunchConfig_t q = {};
            cudaLaunchAttribute qa[1];
            qa[0].id = cudaLaunchAttributeClusterDimension;
            qa[0].val.clusterDim.x = unsigned(s);
            qa[0].val.clusterDim.y = 1;
            qa[0].val.clusterDim.z = 1;
            q.gridDim = dim3(unsigned(s * num_sms));
            q.blockDim = dim3(Cfg::THREADS);
            q.dynamicSmemBytes = Cfg::SMEM;
            q.attrs = qa;
            q.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &q);
            if (e != cudaSuccess)
                return e;
            if (n < 1)
                return cudaErrorInvalidConfiguration;
            // The query counts one CTA per SM for a kernel that holds tensor memory.  Two whose
            // registers, shared and tensor memory fit do share an SM (seen by their SM numbers
            // and times: 192 CTAs on 148 SMs, 44 of them with two at once).
            cache[s].set(dev, n * Cfg::BLOCKS);
        }
    }
    int fit[FEW_MAX_SPLIT + 1];
    fit[0] = 0;
    for (int s = 1; s <= FEW_MAX_SPLIT; ++s)
        fit[s] = cache[s].get(dev);
    CUtensorMap tw, th;
    if (!codes_map(&tw, w, uint64_t(w_rows), uint64_t(a.K), 128))
        return cudaErrorInvalidValue;
    th = tw;  // only used where the tokens' codes are in memory
    if (!Cfg::QUANT && !codes_map(&th, codes, uint64_t(a.sx_rows), uint64_t(a.K), Cfg::NT))
        return cudaErrorInvalidValue;
    // The most items there may be: an expert's rows make whole units but for one, which
    // is the only one where all tokens make no more.  A cluster takes one item at most, so
    // those that split theirs have to cover them all.
    const int64_t pairs = int64_t(a.T) * a.k, whole = a.T <= Cfg::NT ? 0 : pairs / Cfg::NT;
    const int64_t units = Cfg::EXPERTS ? (pairs < a.E ? pairs : a.E) + whole : 1;
    const int64_t items = units * (a.N / 128 / Cfg::RT), slots = fit[1];
    const int split = few_split(items, a.KB, num_sms, fit);
    for (int s = 0; s <= split; ++s)
        a.part_lo[s] = int(int64_t(a.KB) * s / split);
    const uint64_t tiles = uint64_t(a.N / 128 / Cfg::RT);
    a.tiles_inv = tiles == 1 ? 0xFFFFFFFFu : uint32_t(((uint64_t(1) << 32) + tiles - 1) / tiles);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    set_pdl(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(split);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    // an expert CTA walks items; the others have one each
    cfg.gridDim = dim3(unsigned(!Cfg::EXPERTS || split > 1 || items < slots ? items * split : slots));
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, tw, th, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

size_t linear_few_workspace(int T, int64_t K)
{
    // codes, then scales (a small weight does without)
    return T <= FEW_QUANT_TOKENS ? 0 : size_t(T) * K + size_t(T) * (K / 128) * 4;
}

cudaError_t launch_linear_few(const void *x, int T, const uint8_t *qw, const float *sw, void *y,
                              int64_t N, int64_t K, void *workspace, cudaStream_t stream, int num_sms)
{
    FewArgs a = {};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.sw = sw;
    a.y = static_cast<__nv_bfloat16 *>(y);
    a.T = T;
    a.k = 1;
    a.E = 1;
    a.N = int(N);
    a.K = int(K);
    a.KB = int(K / 128);
    if (T <= FEW_QUANT_TOKENS || (T <= FEW_QUANT_TOKENS_SMALL && N * K <= FEW_QUANT_SMALL))
        return run_few<FewCfg<FEW_LINEAR, 16>>(qw, N, nullptr, a, stream, num_sms);
    uint8_t *q = static_cast<uint8_t *>(workspace);
    float *s = reinterpret_cast<float *>(q + size_t(T) * K);
    a.sx = s;
    a.sx_rows = T;
    const cudaError_t e = launch_quant_act(x, T, K, q, s, stream, num_sms);
    if (e != cudaSuccess)
        return e;
    if (T <= 16)
        return run_few<FewCfg<FEW_CODES, 16>>(qw, N, q, a, stream, num_sms);
    return T <= 32 ? run_few<FewCfg<FEW_CODES, 32>>(qw, N, q, a, stream, num_sms)
                   : run_few<FewCfg<FEW_CODES, 64>>(qw, N, q, a, stream, num_sms);
}

// The workspace of the layer: codes and scales of h, each pair's product, counters.
struct FewSpace {
    size_t hs, part, count, bytes;  // the codes come first
    FewSpace(int T, int k, int64_t H, int64_t I)
    {
        const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
        const size_t pairs = size_t(T) * size_t(k);
        hs = up(pairs * size_t(I));
        part = hs + up(pairs * size_t(I / 128) * 4);
        count = part + up(pairs * size_t(H) * 4);
        bytes = count + up(size_t(T) * size_t(H / 128) * 4);
    }
};

size_t moe_few_workspace(int T, int k, int64_t H, int64_t I)
{
    return FewSpace(T, k, H, I).bytes;
}

cudaError_t launch_moe_few(const void *x, int T, const uint8_t *w1, const float *s1,
                           const uint8_t *w2, const float *s2, const int32_t *ids,
                           const float *weights, int k, int E, int64_t H, int64_t I, void *y,
                           void *workspace, cudaStream_t stream, int num_sms)
{
    const FewSpace space(T, k, H, I);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    FewArgs a = {};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.sw = s1;
    a.ids = ids;
    a.weights = weights;
    a.y = static_cast<__nv_bfloat16 *>(y);
    a.hq = ws;
    a.hs = reinterpret_cast<float *>(ws + space.hs);
    a.part = reinterpret_cast<float *>(ws + space.part);
    a.count = reinterpret_cast<int *>(ws + space.count);
    a.T = T;
    a.k = k;
    a.E = E;
    a.N = int(2 * I);
    a.K = int(H);
    a.KB = int(H / 128);
    a.tiles_h = int(H / 128);
    cudaError_t e = T <= 16
        ? run_few<FewCfg<FEW_UP, 16>>(w1, E * 2 * I, nullptr, a, stream, num_sms)
        : run_few<FewCfg<FEW_UP, 32>>(w1, E * 2 * I, nullptr, a, stream, num_sms);
    if (e != cudaSuccess)
        return e;
    a.sw = s2;
    a.N = int(H);
    a.K = int(I);
    a.KB = int(I / 128);
    a.sx = a.hs;
    a.sx_rows = T * k;
    return T <= 16 ? run_few<FewCfg<FEW_DOWN, 16>>(w2, E * H, ws, a, stream, num_sms)
                   : run_few<FewCfg<FEW_DOWN, 32>>(w2, E * H, ws, a, stream, num_sms);
}

cudaError_t read_and_clear_few_error(int *value)
{
    cudaError_t e = cudaMemcpyFromSymbol(value, g_few_error, sizeof(int));
    if (e != cudaSuccess)
        return e;
    if (*value) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_few_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace fp8bw
