// moe_route.cu -- the router of a mixture-of-experts layer: top-k choice with softmax
// weights, the gradient of the logits, and the plan that lays the chosen (token,
// expert) pairs out by expert for the grouped GEMM.
//
// All three are bound by memory latency at small sizes and by issue slots at large
// ones; the bytes they move are small next to the layer's products.
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch_cache.cuh"
#include "moe.cuh"
#include "ptx.cuh"

namespace fp8bw {

constexpr int ROUTE_WARPS = 8;  // one warp per token

// The logits of one row, spread over a warp: register c * V + v of lane l holds expert
// c * 32 * V + l * V + v, so that V contiguous values come from one load.
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// A logit that may be chosen: finite.  +inf counts as the largest finite value, so that
// the softmax stays defined; -inf and NaN mark experts that are not available (-inf here).
__device__ __forceinline__ float usable(float v)
{
    return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY;
}

template <class T, int V, int NV>
__device__ __forceinline__ void load_row(const T *row, int E, int lane, float (&v)[NV])
{
    struct alignas(sizeof(T) * V) Vec { T e[V]; };
#pragma unroll
    for (int c = 0; c < NV / V; ++c) {
        const int at = (c * 32 + lane) * V;
        if (at < E) {  // E is a multiple of V
            const Vec w = *reinterpret_cast<const Vec *>(row + at);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[c * V + i] = usable(to_f32(w.e[i]));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[c * V + i] = -INFINITY;
        }
    }
}

template <int V> __device__ __forceinline__ int expert_of(int i, int lane)
{
    return (i / V * 32 + lane) * V + i % V;
}

// Unsigned key whose order is that of the floats; -0 and +0 get one key, -inf gets 0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return v > -INFINITY ? (u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u)) : 0u;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// weights[t][j], ids[t][j] for the k largest logits of row t, largest first, ties to
// the lowest expert.  One warp per token: k rounds of a warp-wide maximum (redux) over
// each lane's best remaining value; lane j keeps choice j.  Statistics in FP32.
template <class T, int V, int NV>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
moe_route_kernel(const T *__restrict__ logits, int64_t rows, int E, int k, int renorm,
                 float *__restrict__ weights, int32_t *__restrict__ ids)
{
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5); t < rows;
         t += int64_t(gridDim.x) * ROUTE_WARPS) {
        float v[NV];
        load_row<T, V, NV>(logits + t * E, E, lane, v);
        uint32_t left[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            left[i] = order_key(v[i]);
        float mine = -INFINITY, top = 0.0f;
        int my_id = -1;
        for (int j = 0; j < k; ++j) {
            uint32_t best = left[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < NV; ++i)
                if (left[i] > best) {
                    best = left[i];
                    at = i;
                }
            const uint32_t high = __reduce_max_sync(0xffffffffu, best);
            if (high == 0u)  // nothing is left: this choice and the later ones stay empty
                break;
            const uint32_t e = best == high ? uint32_t(expert_of<V>(at, lane)) : 0xFFFFFFFFu;
            const uint32_t first = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first == uint32_t(expert_of<V>(i, lane)))
                    left[i] = 0u;
            const uint32_t u = (high >> 31) ? (high ^ 0x80000000u) : ~high;
            const float val = __uint_as_float(u);
            if (j == 0)
                top = val;
            if (lane == j) {
                mine = val;
                my_id = int(first);
            }
        }
        const float p = my_id >= 0 ? expf(mine - top) : 0.0f;
        float den;
        if (renorm) {
            den = warp_sum(p);
        } else {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                s += v[i] > -INFINITY ? expf(v[i] - top) : 0.0f;
            den = warp_sum(s);
        }
        if (lane < k) {
            weights[t * k + lane] = my_id >= 0 ? p / den : 0.0f;
            ids[t * k + lane] = my_id;
        }
    }
}

// dlogits = direct - p * (sum_j w_j dw_j): direct is w_j dw_j at the chosen experts, p
// the softmax over the chosen experts (renorm, so p = w there and 0 elsewhere) or over
// all.  Every element of the row is written.  A choice with an id outside [0, E) takes
// no part.  One warp per token, in FP32, rounded once to the logits' type.
template <class T, int V, int NV>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
moe_route_bwd_kernel(const float *__restrict__ dweights, const float *__restrict__ weights,
                     const int32_t *__restrict__ ids, const T *__restrict__ logits, int64_t rows,
                     int E, int k, int renorm, T *__restrict__ dlogits)
{
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5); t < rows;
         t += int64_t(gridDim.x) * ROUTE_WARPS) {
        int id = -1;
        float w = 0.0f, dw = 0.0f;
        if (lane < k) {
            id = ids[t * k + lane];
            w = weights[t * k + lane];
            dw = dweights[t * k + lane];
        }
        const bool some = id >= 0 && id < E;
        const float direct = some ? w * dw : 0.0f;
        const float total = warp_sum(direct);
        const float g = renorm ? direct - (some ? w : 0.0f) * total : direct;
        float d[NV];
        if (renorm) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i] = 0.0f;
        } else {
            load_row<T, V, NV>(logits + t * E, E, lane, d);
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                m = fmaxf(m, d[i]);
            m = warp_max(m);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                d[i] = d[i] > -INFINITY ? expf(d[i] - m) : 0.0f;
                s += d[i];
            }
            s = warp_sum(s);
            const float c = s > 0.0f ? -total / s : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i] *= c;
        }
        for (int j = 0; j < k; ++j) {
            const int e = __shfl_sync(0xffffffffu, some ? id : -1, j);
            const float ge = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e == expert_of<V>(i, lane))
                    d[i] += ge;
        }
        struct alignas(sizeof(T) * V) Vec { T e[V]; };
#pragma unroll
        for (int c = 0; c < NV / V; ++c) {
            const int at = (c * 32 + lane) * V;
            if (at < E) {
                Vec o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.e[i] = from_f32<T>(d[c * V + i]);
                *reinterpret_cast<Vec *>(dlogits + t * E + at) = o;
            }
        }
    }
}

// ------------------------------------------------------------------------- plan

// The pairs (t, j), in order p = t * k + j, are cut into `chunks` equal runs, one CTA
// each, and each CTA's run into one run per warp.  Counting the ids of every run
// gives, by prefix sums over warps and chunks, the place at which each run's first pair
// of an expert goes; inside a run a warp ranks 32 pairs at a time by matching ids.  All
// sums are of whole numbers, and a pair's place depends on the ids alone.
constexpr int PLAN_WARPS = 16;
constexpr int PLAN_THREADS = PLAN_WARPS * 32;
constexpr int PLAN_PAIRS = 2048;  // pairs of a chunk, at least
constexpr int PLAN_CHUNKS = 128;

static int plan_chunks(int64_t pairs)
{
    const int64_t c = (pairs + PLAN_PAIRS - 1) / PLAN_PAIRS;
    return int(c < 1 ? 1 : c > PLAN_CHUNKS ? PLAN_CHUNKS : c);
}

struct PlanRun {
    int64_t lo, hi;
    __device__ PlanRun(int64_t pairs, int chunk, int chunks, int warp)
    {
        const int64_t runs = int64_t(chunks) * PLAN_WARPS, r = int64_t(chunk) * PLAN_WARPS + warp;
        const int64_t len = ((pairs + runs - 1) / runs + 31) / 32 * 32;
        lo = min(pairs, r * len);
        hi = min(pairs, lo + len);
    }
};

// Adds each id of the warp's run to cnt[E] (shared, this warp's own); -1 for an id
// outside [0, E).
__device__ __forceinline__ void plan_count(const int32_t *ids, const PlanRun &run, int E, int lane,
                                           int *cnt)
{
    for (int64_t p = run.lo + lane; p < run.hi; p += 32) {
        const int id = ids[p];
        if (id >= 0 && id < E)
            atomicAdd(&cnt[id], 1);
    }
}

__global__ void __launch_bounds__(PLAN_THREADS)
moe_plan_count_kernel(const int32_t *__restrict__ ids, int64_t pairs, int E, int *__restrict__ hist)
{
    extern __shared__ int cnt[];  // [PLAN_WARPS][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < PLAN_WARPS * E; i += PLAN_THREADS)
        cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    plan_count(ids, PlanRun(pairs, blockIdx.x, gridDim.x, warp), E, lane, cnt + warp * E);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS) {
        int s = 0;
        for (int w = 0; w < PLAN_WARPS; ++w)
            s += cnt[w * E + e];
        hist[blockIdx.x * E + e] = s;
    }
}

__global__ void __launch_bounds__(PLAN_THREADS)
moe_plan_place_kernel(const int32_t *__restrict__ ids, int64_t pairs, int E,
                      const int *__restrict__ hist, int64_t rows, int32_t *__restrict__ seg,
                      int32_t *__restrict__ row, int32_t *__restrict__ src)
{
    extern __shared__ int sh[];
    int *cnt = sh;                    // [PLAN_WARPS][E]
    int *total = cnt + PLAN_WARPS * E;  // [E]
    int *before = total + E;          // [E] pairs of the expert in earlier chunks
    int *first = before + E;          // [E + 1] first block of the expert
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = blockIdx.x, chunks = gridDim.x;
    for (int i = threadIdx.x; i < (PLAN_WARPS + 2) * E; i += PLAN_THREADS)
        sh[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const PlanRun run(pairs, chunk, chunks, warp);
    plan_count(ids, run, E, lane, cnt + warp * E);
    if (chunks > 1) {
        // the other chunks' counts: a few chunks per thread and expert, summed in shared memory
        const int parts = max(1, PLAN_THREADS / E);
        for (int i = threadIdx.x; i < parts * E; i += PLAN_THREADS) {
            const int e = i % E, part = i / E;
            int b = 0, s = 0;
            for (int c = part; c < chunks; c += parts) {
                const int h = hist[c * E + e];
                s += h;
                b += c < chunk ? h : 0;
            }
            atomicAdd(&total[e], s);
            atomicAdd(&before[e], b);
        }
    }
    __syncthreads();
    // counts of each warp's run -> where the run's first pair of each expert goes
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS) {
        int s = before[e];
        for (int w = 0; w < PLAN_WARPS; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = s;
            s += c;
        }
        if (chunks == 1)
            total[e] = s;
    }
    __syncthreads();
    if (warp == 0) {  // blocks of each expert, summed over the experts before it
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int b = e < E ? (total[e] + 127) / 128 : 0;
            int s = b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, s, o);
                s += lane >= o ? up : 0;
            }
            if (e < E)
                first[e] = carry + s - b;
            carry += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0)
            first[E] = carry;
    }
    __syncthreads();
    if (chunk == 0)
        for (int e = threadIdx.x; e <= E; e += PLAN_THREADS)
            seg[e] = first[e];
    int *mine = cnt + warp * E;
    for (int64_t p0 = run.lo; p0 < run.hi; p0 += 32) {
        const int64_t p = p0 + lane;
        int id = p < run.hi ? ids[p] : -1;
        if (id < 0 || id >= E)
            id = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        int at = 0;
        if (id >= 0)
            at = mine[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (id >= 0 && lane == 31 - __clz(same))
            mine[id] = at + 1;
        __syncwarp();
        if (p < run.hi) {
            const int64_t r = id >= 0 ? int64_t(first[id]) * 128 + at : -1;
            row[p] = int32_t(r);
            if (r >= 0)
                src[r] = int32_t(p);
        }
    }
    // rows that no pair takes: the rest of each expert's last block, and all behind the last
    for (int e = chunk * PLAN_WARPS + warp; e < E; e += chunks * PLAN_WARPS)
        for (int64_t r = int64_t(first[e]) * 128 + total[e] + lane; r < int64_t(first[e + 1]) * 128;
             r += 32)
            src[r] = -1;
    for (int64_t r = int64_t(first[E]) * 128 + int64_t(chunk) * PLAN_THREADS + threadIdx.x; r < rows;
         r += int64_t(chunks) * PLAN_THREADS)
        src[r] = -1;
}

// ------------------------------------------------------------------- host side

template <class K, class... A>
static cudaError_t launch(K kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    set_pdl(at[0]);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Calls f with the row layout as types: V values per load, NV values per lane.
template <class T, class F> static cudaError_t with_layout(int E, F f)
{
    constexpr int W = 16 / sizeof(T);
    struct L1_4 { enum { V = 1, NV = 4 }; };
    struct L1_8 { enum { V = 1, NV = 8 }; };
    struct L1_32 { enum { V = 1, NV = 32 }; };
    struct LW_W { enum { V = W, NV = W }; };
    struct LW_2W { enum { V = W, NV = 2 * W }; };
    struct LW_32 { enum { V = W, NV = 32 }; };
    if (E % W == 0) {  // rows of whole 16-byte pieces
        if (E <= 32 * W)
            return f(LW_W());
        return E <= 64 * W ? f(LW_2W()) : f(LW_32());
    }
    if (E <= 128)
        return f(L1_4());
    return E <= 256 ? f(L1_8()) : f(L1_32());
}

static dim3 route_grid(int64_t T, int num_sms)
{
    const int64_t blocks = (T + ROUTE_WARPS - 1) / ROUTE_WARPS;
    const int64_t most = int64_t(num_sms) * (2048 / (ROUTE_WARPS * 32));
    return dim3(unsigned(blocks < most ? blocks : most));
}

template <class T>
static cudaError_t route(const void *logits, int64_t rows, int E, int k, bool renorm, float *weights,
                         int32_t *ids, cudaStream_t stream, int num_sms)
{
    return with_layout<T>(E, [&](auto l) {
        using L = decltype(l);
        return launch(moe_route_kernel<T, L::V, L::NV>, route_grid(rows, num_sms), ROUTE_WARPS * 32,
                      0, stream, static_cast<const T *>(logits), rows, E, k, int(renorm), weights,
                      ids);
    });
}

template <class T>
static cudaError_t route_bwd(const float *dweights, const float *weights, const int32_t *ids,
                             const void *logits, int64_t rows, int E, int k, bool renorm,
                             void *dlogits, cudaStream_t stream, int num_sms)
{
    return with_layout<T>(E, [&](auto l) {
        using L = decltype(l);
        return launch(moe_route_bwd_kernel<T, L::V, L::NV>, route_grid(rows, num_sms),
                      ROUTE_WARPS * 32, 0, stream, dweights, weights, ids,
                      static_cast<const T *>(logits), rows, E, k, int(renorm),
                      static_cast<T *>(dlogits));
    });
}

cudaError_t launch_moe_route(const void *logits, bool bf16, int64_t T, int E, int k, bool renorm,
                             float *weights, int32_t *ids, cudaStream_t stream, int num_sms)
{
    return bf16 ? route<__nv_bfloat16>(logits, T, E, k, renorm, weights, ids, stream, num_sms)
                : route<float>(logits, T, E, k, renorm, weights, ids, stream, num_sms);
}

cudaError_t launch_moe_route_bwd(const float *dweights, const float *weights, const int32_t *ids,
                                 const void *logits, bool bf16, int64_t T, int E, int k,
                                 bool renorm, void *dlogits, cudaStream_t stream, int num_sms)
{
    return bf16 ? route_bwd<__nv_bfloat16>(dweights, weights, ids, logits, T, E, k, renorm, dlogits,
                                           stream, num_sms)
                : route_bwd<float>(dweights, weights, ids, logits, T, E, k, renorm, dlogits, stream,
                                   num_sms);
}

int64_t moe_plan_rows(int64_t T, int k, int E)
{
    const int64_t pairs = T * k;
    return (pairs + 127 * (pairs < E ? pairs : int64_t(E))) / 128 * 128;
}

size_t moe_plan_workspace(int64_t T, int k, int E)
{
    return size_t(plan_chunks(T * k)) * size_t(E) * sizeof(int);
}

cudaError_t launch_moe_plan(const int32_t *ids, int64_t T, int k, int E, int32_t *seg,
                            int32_t *row, int32_t *src, void *workspace, cudaStream_t stream)
{
    const int64_t pairs = T * k;
    const int chunks = plan_chunks(pairs);
    const size_t count_smem = size_t(PLAN_WARPS) * E * sizeof(int);
    const size_t place_smem = count_smem + (3 * size_t(E) + 1) * sizeof(int);
    if (place_smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(
            moe_plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(moe_plan_count_kernel,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
        if (e != cudaSuccess)
            return e;
    }
    int *hist = static_cast<int *>(workspace);
    if (chunks > 1) {
        cudaError_t e = launch(moe_plan_count_kernel, dim3(chunks), PLAN_THREADS, count_smem, stream,
                               ids, pairs, E, hist);
        if (e != cudaSuccess)
            return e;
    }
    return launch(moe_plan_place_kernel, dim3(chunks), PLAN_THREADS, place_smem, stream, ids, pairs,
                  E, static_cast<const int *>(hist), moe_plan_rows(T, k, E), seg, row, src);
}

} // namespace fp8bw
