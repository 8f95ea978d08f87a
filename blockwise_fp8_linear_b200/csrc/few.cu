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
// shared memory without passing through registers.  One CTA takes a tile of 128
// weight rows (up: 128 gate rows and the 128 up rows beside them) and one part of the
// reduction; the CTAs of a cluster split the reduction, so that a small weight still
// keeps most SMs reading, and join their FP32 sums through distributed shared memory in
// a fixed order.
//
//   warps 0..3  promotion: partial sums of a 128-block from TMEM (thread = weight row),
//               times weight scale x token scale, into FP32 sums in registers
//   warp 4      TMA producer: weight tiles (down: also the codes of h)
//   warp 5      MMA issuer
//   warps 6..   linear, up: quantize the tokens' 1x128 groups of this block into shared
//               memory (the arithmetic of fp8_quant_act); down: load the scales of h
//
// An expert's rows: the tokens that chose it, in token order.  Every CTA works them out
// from the ids, which are at most 2048 numbers.  Every wait is bounded.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch_cache.cuh"
#include "moe.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"
#include "tensor_map.cuh"

namespace fp8bw {

__device__ int g_few_error;  // first error code of a bounded wait in these kernels
constexpr uint64_t FEW_WAIT_NS = 1000000000ull;
constexpr uint64_t FEW_DRAIN_NS = 20000000ull;
enum : int { FERR_PRODUCER = 31, FERR_MMA_FULL = 32, FERR_MMA_TEMPTY = 33, FERR_PROMO = 34, FERR_ACT = 35 };

enum : int { FEW_LINEAR = 0, FEW_UP = 1, FEW_DOWN = 2 };

struct FewArgs {
    const __nv_bfloat16 *x;  // [T][K] (linear, up)
    const float *sw;         // weight block scales [E][N/128][K/128]
    const int32_t *ids;      // [T][k] (up, down)
    const float *weights;    // [T][k] (down)
    __nv_bfloat16 *y;        // [T][N] (linear, down)
    uint8_t *hq;             // [T*k][I] codes of h, rows by expert (up writes, down reads)
    float *hs;               // [I/128][T*k] their scales
    float *part;             // [T*k][H] products of each pair (down)
    int *count;              // [T][H/128] experts of the token that are done (down)
    int T, k, E;
    int N, K, KB;            // rows and columns of one expert's weight, K / 128
    int tiles_h;             // H / 128 (up clears the counters)
};

template <int KIND_, int NT_>
struct FewCfg {
    static constexpr int KIND = KIND_;
    static constexpr int NT = NT_;                      // token columns of the MMA
    static constexpr int RT = KIND == FEW_UP ? 2 : 1;   // 128-row tiles: gate and up, or one
    static constexpr int W_BYTES = RT * 128 * 128;
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    // Two CTAs share an SM, so one's prologue and epilogue run under the other's loads;
    // up with 64 columns keeps 128 sums per thread and has an SM to itself.
    static constexpr int BLOCKS = RT * NT <= 64 ? 2 : 1;
    static constexpr int STAGES = 216 / BLOCKS * 1024 / STAGE_BYTES;
    static constexpr int ACT_WARPS = KIND == FEW_DOWN ? 1 : 4;
    static constexpr int THREADS = (6 + ACT_WARPS) * 32;
    static constexpr int NBUF = 2;
    static constexpr int TMEM_COLS = NBUF * RT * NT;    // 32 .. 256, a power of two
    static constexpr int RED_BYTES = RT * NT * 128 * 4;  // the joined sums reuse the stages
    static constexpr int XS_OFF = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFF = XS_OFF + STAGES * NT * 4;
    static constexpr int SMEM = 1024 + BAR_OFF + (2 * STAGES + 2 * NBUF) * 8 + 16;
    static_assert(RED_BYTES <= STAGES * STAGE_BYTES, "the joined sums must fit the stages");
    static_assert(TMEM_COLS >= 32 && TMEM_COLS * BLOCKS <= 512, "tensor memory of an SM");
    // 228 KB per SM, 1 KB of it reserved per CTA; FewPlan is static
    static_assert((SMEM + 1024 + 512) * BLOCKS <= 228 * 1024, "shared memory of an SM");
};

// What one CTA of the expert kernels works on: the expert, its rows and where they stand.
struct FewItem {
    int expert;  // -1: no such item
    int rows;
    int base;    // first row of the expert in the order by (expert, token)
};

struct FewPlan {
    uint32_t hit[32];               // experts that some token chose
    uint32_t mask[2];               // tokens of this expert
    int16_t row_pair[kFewMaxTokens];  // pair (token * k + choice) of each row
    uint8_t row_token[kFewMaxTokens];
    int expert, base;
};

// Expert number `slot` among those that some token chose, its tokens in order, and how
// many (expert, token) rows the experts before it have.  A token that names an expert
// twice counts once, at its first choice.  All threads of the CTA call it; `id` is
// scratch in shared memory, one entry per pair.
__device__ __forceinline__ FewItem few_plan(FewPlan &p, int16_t *id, const int32_t *ids, int T, int k,
                                            int E, int slot)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 32)
        p.hit[tid] = 0;
    if (tid == 0) {
        p.expert = -1;
        p.base = 0;
    }
    __syncthreads();
    for (int i = tid; i < T * k; i += blockDim.x) {
        const int v = ids[i];
        const bool ok = v >= 0 && v < E;
        id[i] = int16_t(ok ? v : -1);
        if (ok)
            atomicOr(&p.hit[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t word = p.hit[lane];
        const int n = __popc(word);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, before, o);
            before += lane >= o ? up : 0;
        }
        before -= n;
        if (slot >= before && slot < before + n) {
            for (int i = before; i < slot; ++i)
                word &= word - 1;
            p.expert = lane * 32 + __ffs(word) - 1;
        }
    }
    __syncthreads();
    const int e = p.expert;
    if (e < 0)
        return {-1, 0, 0};
    int earlier = 0;
    for (int i = tid; i < T * k; i += blockDim.x) {
        const int v = id[i];
        if (v >= 0 && v < e) {
            bool first = true;
            for (int q = i / k * k; q < i; ++q)
                first = first && id[q] != v;
            earlier += first ? 1 : 0;
        }
    }
    earlier = __reduce_add_sync(0xffffffffu, earlier);
    if (lane == 0 && earlier)
        atomicAdd(&p.base, earlier);
    int choice = -1;
    if (tid < kFewMaxTokens) {
        if (tid < T)
            for (int j = k - 1; j >= 0; --j)
                if (id[tid * k + j] == e)
                    choice = j;
        const uint32_t m = __ballot_sync(0xffffffffu, choice >= 0);
        if (lane == 0)
            p.mask[warp] = m;
    }
    __syncthreads();
    if (choice >= 0) {
        const int r = __popc(p.mask[warp] & ((1u << lane) - 1u)) + (warp ? __popc(p.mask[0]) : 0);
        p.row_token[r] = uint8_t(tid);
        p.row_pair[r] = int16_t(tid * k + choice);
    }
    __syncthreads();
    return {e, __popc(p.mask[0]) + __popc(p.mask[1]), p.base};
}

__device__ __forceinline__ uint2 bf16x4(float4 v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// This lane's choice of token t (lane j: choice j): its id, -1 where a lower choice names
// the same expert, and the weight of all choices that name it, summed in their order.
__device__ __forceinline__ int few_choice(const FewArgs &a, int t, int lane, float &weight)
{
    int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    if (id < 0 || id >= a.E)
        id = -1;
    const float w = lane < a.k ? a.weights[t * a.k + lane] : 0.0f;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    weight = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        if ((same >> j) & 1u)
            weight += wj;
    }
    return (id >= 0 && __ffs(same) - 1 == lane) ? id : -1;
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
    float *xs = reinterpret_cast<float *>(smem + Cfg::XS_OFF);       // [STAGES][NT] token scales
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + NBUF;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tempty + NBUF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    __shared__ FewPlan plan;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = int(cluster_ctarank()), split = int(cluster_nctarank());
    const int tile = int(blockIdx.x) / split;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1 + Cfg::ACT_WARPS);
            mbar_init(&empty[s], 1 + 4);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 4);
        }
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmW);
    }
    if (warp == 5) {
        tmem_alloc<1>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<1>();
    }
    if (KIND != FEW_DOWN) {
        // columns without a token stay zero for good
        for (int i = tid; i < STAGES * Cfg::X_BYTES / 16; i += Cfg::THREADS) {
            const int s = i / (Cfg::X_BYTES / 16), o = i % (Cfg::X_BYTES / 16);
            *reinterpret_cast<uint4 *>(smem + s * Cfg::STAGE_BYTES + Cfg::W_BYTES + 16 * o) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // The tensor memory is held before a dependent kernel may start: one that started
    // first and took it would wait for this one, which would wait for it.
    FewItem item = {0, a.T, 0};
    if (KIND != FEW_DOWN) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (KIND == FEW_UP && blockIdx.y == 0)
        for (int i = int(blockIdx.x) * Cfg::THREADS + tid; i < a.T * a.tiles_h;
             i += int(gridDim.x) * Cfg::THREADS)
            a.count[i] = 0;
    // down: the ids (like the weights) were complete before the up kernel began, which
    // waited for its predecessor before it let this one start
    if (KIND != FEW_LINEAR) {
        // its scratch is the first stage's weight tile, which the copies below overwrite
        item = few_plan(plan, reinterpret_cast<int16_t *>(smem), a.ids, a.T, a.k, a.E,
                        int(blockIdx.y));
        fence_proxy_async_smem();
        __syncthreads();
    }

    const int lo = a.KB * rank / split, hi = a.KB * (rank + 1) / split;
    const int nkb = item.expert < 0 ? 0 : hi - lo;
    const int n_tiles = a.N / 128;
    const int wrow = item.expert * a.N + tile * 128;  // up: of the gate rows

    if (warp < 4) {
        // ------------------------------------------------------------- promotion
        float acc[RT][NT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < NT; ++c)
                acc[r][c] = 0.0f;
        if (nkb > 0) {
            const float *sw[RT];
            float next[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                sw[r] = a.sw + (size_t(item.expert) * n_tiles + tile + r * (n_tiles / 2)) * a.KB + lo;
                next[r] = __ldg(sw[r]);
            }
            for (int i = 0; i < nkb; ++i) {
                const int s = i % STAGES, b = i % NBUF;
                float cur[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    cur[r] = next[r];
                    if (i + 1 < nkb)
                        next[r] = __ldg(sw[r] + i + 1);
                }
                // the stage's full barrier cannot run ahead: it waits for this warp below
                const bool ok =
                    mbar_wait_bounded(&full[s], uint32_t(i / STAGES) & 1u, abort_flag, &g_few_error,
                                      FERR_PROMO, FEW_WAIT_NS) &&
                    mbar_wait_bounded(&tfull[b], uint32_t(i / NBUF) & 1u, abort_flag, &g_few_error,
                                      FERR_PROMO, FEW_WAIT_NS);
                if (!__all_sync(0xffffffffu, ok))
                    break;
                tc_fence_after();
                const uint32_t taddr =
                    tmem_base + (uint32_t(warp * 32) << 16) + uint32_t(b * RT * NT);
                const float4 *xs4 = reinterpret_cast<const float4 *>(xs + s * NT);
                // 16 columns at a time: the sums already take RT x NT registers
#pragma unroll
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    uint32_t v[RT][16];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        tmem_ld_32x32b_x16(taddr + uint32_t(r * NT + c0), v[r]);
                    tmem_wait_ld();
                    if (c0 + 16 == NT) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&tempty[b]);
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 x4 = xs4[(c0 + c) / 4];
                        const float xc[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                acc[r][c0 + c + q] = fmaf(__uint_as_float(v[r][c + q]),
                                                          cur[r] * xc[q], acc[r][c0 + c + q]);
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&empty[s]);
            }
            // Every product of this CTA is done (the last buffer was full), so no copy or
            // MMA touches the stages any more: they take the sums, [RT][NT][128].
            float *red = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (c < item.rows)
                        red[(r * NT + c) * 128 + tid] = acc[r][c];
        }
    } else if (warp == 4) {
        // -------------------------------------------------------------- producer
        if (lane == 0 && nkb > 0) {
            const int bytes = Cfg::W_BYTES + (KIND == FEW_DOWN ? Cfg::X_BYTES : 0);
            int ahead = 0;  // down: stages whose weights were asked for before the wait
            if (KIND == FEW_DOWN) {
                ahead = min(STAGES, nkb);
                for (int i = 0; i < ahead; ++i) {
                    mbar_arrive_expect_tx(&full[i], bytes);
                    tma_load_2d(smem + i * Cfg::STAGE_BYTES, &tmW, &full[i], (lo + i) * 128, wrow);
                }
                pdl_wait();
                pdl_launch_dependents();
            }
            for (int i = 0; i < nkb; ++i) {
                const int s = i % STAGES;
                uint8_t *sw = smem + s * Cfg::STAGE_BYTES;
                if (i >= ahead) {
                    if (!mbar_wait_bounded(&empty[s], (uint32_t(i / STAGES) & 1u) ^ 1u, abort_flag,
                                           &g_few_error, FERR_PRODUCER, FEW_WAIT_NS))
                        break;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    tma_load_2d(sw, &tmW, &full[s], (lo + i) * 128, wrow);
                    if (KIND == FEW_UP)
                        tma_load_2d(sw + 128 * 128, &tmW, &full[s], (lo + i) * 128, wrow + a.N / 2);
                }
                if (KIND == FEW_DOWN)
                    tma_load_2d(sw + Cfg::W_BYTES, &tmH, &full[s], (lo + i) * 128, item.base);
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t idesc = make_idesc_e4m3(128, NT, 0);
            for (int i = 0; i < nkb; ++i) {
                const int s = i % STAGES, b = i % NBUF;
                if (!mbar_spin_bounded(&full[s], uint32_t(i / STAGES) & 1u, abort_flag, &g_few_error,
                                       FERR_MMA_FULL, FEW_WAIT_NS) ||
                    !mbar_spin_bounded(&tempty[b], (uint32_t(i / NBUF) & 1u) ^ 1u, abort_flag,
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
                mma_commit(&empty[s]);
                mma_commit(&tfull[b]);
            }
        }
    } else if (KIND != FEW_DOWN) {
        // -------------------------------------------- quantize the tokens' groups
        // Half-warp w takes rows w, w + 8, ...; lane `sub` of it 8 neighbouring values.
        const int sub = lane & 15, first = (warp - 6) * 2;
        const int row0 = first + (lane >> 4);
        constexpr int ROWS = NT / 8;
        const uint4 *x4 = reinterpret_cast<const uint4 *>(a.x);
        int src[ROWS];  // in pieces of 8 values; -1: no row
        uint4 v[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int r = row0 + 8 * q;
            const int t = KIND == FEW_LINEAR ? r : (r < item.rows ? int(plan.row_token[r]) : 0);
            src[q] = r < item.rows ? t * (a.K / 8) + lo * 16 + sub : -1;
            v[q] = nkb > 0 && src[q] >= 0 ? __ldg(x4 + src[q]) : make_uint4(0u, 0u, 0u, 0u);
        }
        for (int i = 0; i < nkb; ++i) {
            const int s = i % STAGES;
            const bool ok = mbar_wait_bounded(&empty[s], (uint32_t(i / STAGES) & 1u) ^ 1u, abort_flag,
                                              &g_few_error, FERR_ACT, FEW_WAIT_NS);
            if (!__all_sync(0xffffffffu, ok))
                break;
            uint8_t *sx = smem + s * Cfg::STAGE_BYTES + Cfg::W_BYTES;
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                if (first + 8 * q >= item.rows)  // neither half-warp has a row
                    break;
                const int r = row0 + 8 * q;
                const uint4 w = v[q];
                if (src[q] >= 0 && i + 1 < nkb)  // the next block's values are under way meanwhile
                    v[q] = __ldg(x4 + src[q] + (i + 1) * 16);
                uint32_t m2 = __vmaxu2(absmax2(w.x, w.y), absmax2(w.z, w.w));
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1)
                    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
                const float amax = halves_max_to_float(m2);
                const float sc = scale_of_amax(amax);
                if (r < item.rows) {
                    const uint2 codes = amax != 0.0f ? quant8(w, GroupDiv(sc)) : make_uint2(0u, 0u);
                    *reinterpret_cast<uint2 *>(sx + r * 128 + (((sub >> 1) ^ (r & 7)) << 4) +
                                               (sub & 1) * 8) = codes;
                    if (sub == 0)
                        xs[s * NT + r] = sc;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[s]);
        }
    } else {
        // ------------------------------------------------------- scales of h (down)
        pdl_wait();
        for (int i = 0; i < nkb; ++i) {
            const int s = i % STAGES;
            const bool ok = mbar_wait_bounded(&empty[s], (uint32_t(i / STAGES) & 1u) ^ 1u, abort_flag,
                                              &g_few_error, FERR_ACT, FEW_WAIT_NS);
            if (!__all_sync(0xffffffffu, ok))
                break;
            for (int r = lane; r < item.rows; r += 32)
                xs[s * NT + r] = a.hs[size_t(lo + i) * (a.T * a.k) + item.base + r];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[s]);
        }
    }
    if (KIND == FEW_DOWN)
        pdl_wait();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // give copies and MMAs still in flight time to land before the memory is released
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < FEW_DRAIN_NS) {
        }
    }
    if (split > 1)
        cluster_sync();

    // ------------------------------------------------- join the parts, finish the rows
    // One warp per row; lane l has columns 4 l .. 4 l + 3 of the tile.
    const uint32_t red0 = smem_u32(smem);
    for (int r = rank + split * warp; r < item.rows && item.expert >= 0; r += split * WARPS) {
        float4 sum[RT];
#pragma unroll
        for (int q = 0; q < RT; ++q) {
            sum[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t at = red0 + uint32_t(((q * NT + r) * 128 + 4 * lane) * 4);
            for (int p = 0; p < split; ++p) {
                const float4 v = ld_cluster_v4(mapa_shared(at, uint32_t(p)));
                sum[q].x += v.x;
                sum[q].y += v.y;
                sum[q].z += v.z;
                sum[q].w += v.w;
            }
        }
        if (KIND == FEW_LINEAR) {
            *reinterpret_cast<uint2 *>(a.y + size_t(r) * a.N + tile * 128 + 4 * lane) = bf16x4(sum[0]);
        } else if (KIND == FEW_UP) {
            const float g[4] = {sum[0].x, sum[0].y, sum[0].z, sum[0].w};
            const float u[4] = {sum[RT - 1].x, sum[RT - 1].y, sum[RT - 1].z, sum[RT - 1].w};
            float h[4], amax = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h[q] = g[q] / (1.0f + expf(-g[q])) * u[q];
                amax = fmaxf(amax, fabsf(h[q]));
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // h is kept in FP32 up to its one rounding onto E4M3
            const float sc = __fdiv_rn(amax, 448.0f);
            uint32_t codes = 0u;
            if (sc != 0.0f)
                codes = cvt_e4m3x2(__fdiv_rn(h[0], sc), __fdiv_rn(h[1], sc)) |
                        (cvt_e4m3x2(__fdiv_rn(h[2], sc), __fdiv_rn(h[3], sc)) << 16);
            const size_t row = size_t(item.base + r);
            *reinterpret_cast<uint32_t *>(a.hq + row * (a.N / 2) + tile * 128 + 4 * lane) = codes;
            if (lane == 0)
                a.hs[size_t(tile) * (a.T * a.k) + row] = sc;
        } else {
            // The pair's product goes to memory; the warp that brings a token's last one
            // adds them all, in the order of the choices.
            const int t = plan.row_token[r];
            const size_t col = size_t(tile) * 128 + 4 * lane;
            *reinterpret_cast<float4 *>(a.part + size_t(plan.row_pair[r]) * a.N + col) = sum[0];
            float w;
            const int id = few_choice(a, t, lane, w);
            const uint32_t live = __ballot_sync(0xffffffffu, id >= 0);
            __threadfence();
            __syncwarp();
            int done = 0;
            if (lane == 0)
                done = atomicAdd(&a.count[t * n_tiles + tile], 1) + 1;
            done = __shfl_sync(0xffffffffu, done, 0);
            if (done == __popc(live)) {
                __threadfence();
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int j = 0; j < a.k; ++j) {
                    if (!((live >> j) & 1u))
                        continue;
                    const float wj = __shfl_sync(0xffffffffu, w, j);
                    const float4 v = __ldcg(
                        reinterpret_cast<const float4 *>(a.part + size_t(t * a.k + j) * a.N + col));
                    y.x = fmaf(wj, v.x, y.x);
                    y.y = fmaf(wj, v.y, y.y);
                    y.z = fmaf(wj, v.z, y.z);
                    y.w = fmaf(wj, v.w, y.w);
                }
                *reinterpret_cast<uint2 *>(a.y + size_t(t) * a.N + col) = bf16x4(y);
            }
        }
    }
    if (KIND == FEW_DOWN && blockIdx.y == 0 && rank == 0) {
        // tokens that chose no expert
        for (int t = warp; t < a.T; t += WARPS) {
            float w;
            if (!__any_sync(0xffffffffu, few_choice(a, t, lane, w) >= 0))
                *reinterpret_cast<uint2 *>(a.y + size_t(t) * a.N + tile * 128 + 4 * lane) =
                    make_uint2(0u, 0u);
        }
    }
    if (split > 1)
        cluster_sync();  // no peer reads this CTA's sums any more
    else
        __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------------------- host side

// CTAs per tile: the reduction is split until the tiles fill the GPU, with two blocks
// of 128 left for each CTA at least.
static int few_split(int64_t items, int64_t KB, int num_sms)
{
    int s = 1;
    while (s < 8 && items * s * 2 <= 2 * num_sms && KB >= 4 * s)
        s *= 2;
    return s;
}

template <class Cfg>
static cudaError_t run_few(const uint8_t *w, int64_t w_rows, const uint8_t *hq, const FewArgs &a,
                           int64_t tiles, int64_t slots, cudaStream_t stream, int num_sms)
{
    auto kern = few_kernel<Cfg>;
    static LaunchCache cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (cache.get(dev) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
        if (e != cudaSuccess)
            return e;
        cache.set(dev, 1);
    }
    CUtensorMap tw, th;
    if (!codes_map(&tw, w, uint64_t(w_rows), uint64_t(a.K), 128))
        return cudaErrorInvalidValue;
    th = tw;  // not used but by down
    if (Cfg::KIND == FEW_DOWN && !codes_map(&th, hq, uint64_t(a.T) * a.k, uint64_t(a.K), Cfg::NT))
        return cudaErrorInvalidValue;
    const int split = few_split(tiles * slots, a.KB, num_sms);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    set_pdl(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(split);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(tiles * split), unsigned(slots));
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, tw, th, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int KIND>
static cudaError_t run_few_kind(const uint8_t *w, int64_t w_rows, const uint8_t *hq,
                                const FewArgs &a, int64_t tiles, int64_t slots, cudaStream_t stream,
                                int num_sms)
{
    if (a.T <= 16)
        return run_few<FewCfg<KIND, 16>>(w, w_rows, hq, a, tiles, slots, stream, num_sms);
    if (a.T <= 32)
        return run_few<FewCfg<KIND, 32>>(w, w_rows, hq, a, tiles, slots, stream, num_sms);
    return run_few<FewCfg<KIND, 64>>(w, w_rows, hq, a, tiles, slots, stream, num_sms);
}

cudaError_t launch_linear_few(const void *x, int T, const uint8_t *qw, const float *sw, void *y,
                              int64_t N, int64_t K, cudaStream_t stream, int num_sms)
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
    return run_few_kind<FEW_LINEAR>(qw, N, nullptr, a, N / 128, 1, stream, num_sms);
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
    const int64_t slots = int64_t(T) * k < E ? int64_t(T) * k : E;  // experts that can be hit
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
    cudaError_t e = run_few_kind<FEW_UP>(w1, E * 2 * I, ws, a, I / 128, slots, stream, num_sms);
    if (e != cudaSuccess)
        return e;
    a.sw = s2;
    a.N = int(H);
    a.K = int(I);
    a.KB = int(I / 128);
    return run_few_kind<FEW_DOWN>(w2, E * H, ws, a, H / 128, slots, stream, num_sms);
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
