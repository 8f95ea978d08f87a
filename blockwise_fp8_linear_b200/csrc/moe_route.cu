// moe_route.cu -- the router of a mixture-of-experts layer: top-k choice with softmax
// weights, the gradient of the logits, and the plan that lays the chosen (token,
// expert) pairs out by expert for the grouped GEMM.
//
// All three are bound by latency at small sizes and by issue slots at large ones; the
// bytes they move are small next to the layer's products.
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

// A logit that may be chosen: finite.  +inf counts as the type's largest finite value, so
// that the softmax stays defined; -inf and NaN mark experts that are not available (-inf
// here).
template <class T> __device__ __forceinline__ float usable(float v)
{
    const float most = sizeof(T) == 2 ? __uint_as_float(0x7F7F0000u) : FLT_MAX;
    return v > -INFINITY ? fminf(v, most) : -INFINITY;
}

// Rows with +inf or NaN among their logits are rare: one vote finds them, and only they
// pay for usable() (-inf goes its way without).
template <class T, int NV> __device__ __forceinline__ void make_usable(float (&v)[NV])
{
    bool plain = true;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        plain = plain && v[i] < INFINITY;
    if (!__all_sync(0xffffffffu, plain)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = usable<T>(v[i]);
    }
}

// V neighbouring logits in one load: one of them, or 16 bytes.
template <class T, int V> struct Piece;
template <class T> struct Piece<T, 1> {
    T e;
    __device__ __forceinline__ float get(int) const { return to_f32(e); }
    __device__ __forceinline__ static Piece pack(const float *v) { return {from_f32<T>(v[0])}; }
};
template <> struct Piece<float, 4> {
    float4 e;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? e.x : i == 1 ? e.y : i == 2 ? e.z : e.w; }
    __device__ __forceinline__ static Piece pack(const float *v) { return {make_float4(v[0], v[1], v[2], v[3])}; }
};
template <> struct Piece<__nv_bfloat16, 8> {
    uint4 e;
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = i < 2 ? e.x : i < 4 ? e.y : i < 6 ? e.z : e.w;
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
    __device__ __forceinline__ static Piece pack(const float *v)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return {make_uint4(w[0], w[1], w[2], w[3])};
    }
};

// The row as it is loaded (so that the next row's can be under way) and its values.
template <class T, int V, int NV> struct Row {
    Piece<T, V> raw[NV / V];
    __device__ __forceinline__ void load(const T *row, int E, int lane)
    {
#pragma unroll
        for (int c = 0; c < NV / V; ++c) {
            const int at = (c * 32 + lane) * V;
            if (at < E)  // E is a multiple of V
                raw[c] = *reinterpret_cast<const Piece<T, V> *>(row + at);
        }
    }
    __device__ __forceinline__ void values(int E, int lane, float (&v)[NV]) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = (i / V * 32 + lane) * V < E ? raw[i / V].get(i % V) : -INFINITY;
    }
    __device__ __forceinline__ static void copy(T *to, const T *from, int E, int lane)
    {
#pragma unroll
        for (int c = 0; c < NV / V; ++c) {
            const int at = (c * 32 + lane) * V;
            if (at < E)
                *reinterpret_cast<Piece<T, V> *>(to + at) = *reinterpret_cast<const Piece<T, V> *>(from + at);
        }
    }
    __device__ __forceinline__ static void store(T *row, int E, int lane, const float (&v)[NV])
    {
#pragma unroll
        for (int c = 0; c < NV / V; ++c) {
            const int at = (c * 32 + lane) * V;
            if (at < E)
                *reinterpret_cast<Piece<T, V> *>(row + at) = Piece<T, V>::pack(v + c * V);
        }
    }
};

// (register i of a lane is as many experts after its register 0 as in lane 0)
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

// The float of an order key other than 0.
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float((key >> 31) ? (key ^ 0x80000000u) : ~key);
}

// exp(d) for d <= 0 by the hardware's base-2 exponential (2 ulp; the product's rounding
// adds |d| 2^-24).  -inf gives 0.
__device__ __forceinline__ float exp_neg(float d)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * 1.44269504088896341f));
    return r;
}

// The k largest logits of a row, each lane's registers as in Row; a lane's register holds a
// word whose order is theirs.  Nothing has to be taken out between two rounds: relative
// to the last maximum, counting down modulo 2^32, what is below it comes before what is
// not.  Where nothing is below it, the count wraps and `last` climbs back to the largest
// word: a round that does not lower `last` has found nothing.
template <int NV> struct RowWords {
    uint32_t word[NV], last;
    // the next round's maximum distance, and this lane's
    __device__ __forceinline__ uint32_t descend(uint32_t &mine)
    {
        mine = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            mine = max(mine, word[i] - last);
        const uint32_t far = __reduce_max_sync(0xffffffffu, mine);
        last += far;
        return far;
    }
};

// choose() gives lane j the key of choice j (0: none), and every lane that of the first.
// Lane j has its id where OWN_ID is set; otherwise choose() has stored the row's ids.
//
// BF16 logits: value and expert fit one word, (16-bit order key, ~expert), so that words
// are distinct and one warp-wide maximum (redux) finds both.
template <class T, int V, int NV> struct RowTop : RowWords<NV> {
    static constexpr bool OWN_ID = true;
    __device__ __forceinline__ int choose(const float (&v)[NV], int k, int lane, int32_t *,
                                          uint32_t &key, uint32_t &top)
    {
        this->last = 0u;
        const uint32_t first = 0xFFFFu - uint32_t(expert_of<V>(0, lane));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t u = __float_as_uint(__fadd_rn(v[i], 0.0f));
            const uint32_t order = u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
            this->word[i] = (order & 0xFFFF0000u) | (first - uint32_t(expert_of<V>(i, 0)));
        }
        uint32_t mine = next(), top_word = mine;  // lane j: word of choice j, in the end
        int left = 1;
        for (int j = 1; j < k; ++j) {
            const uint32_t w = next();
            if (w == 0u)
                break;
            mine = lane >= j ? w : mine;
            left = j + 1;
        }
        top = key_of(top_word);
        key = lane < left ? key_of(mine) : 0u;
        return key ? int(0xFFFFu - (mine & 0xFFFFu)) : -1;
    }
    // The next word, 0 when none is left (-inf has the lowest key, 0x007F).
    __device__ __forceinline__ uint32_t next()
    {
        uint32_t unused;
        this->descend(unused);
        return this->last >= 0x00800000u ? this->last : 0u;
    }
    // (the low half of a BF16 value's key is all its sign's)
    __device__ __forceinline__ static uint32_t key_of(uint32_t w)
    {
        return w == 0u ? 0u : (w >> 31) ? w & 0xFFFF0000u : w | 0xFFFFu;
    }
};

// FP32 logits: the rounds find the k largest keys, each lane noting the rounds that it won;
// which register it was is looked up afterwards, once per lane and win (two or three times,
// in place of k).  Equal logits among the choices show in there being more registers of at
// least the last key than rounds (as there are, too, where a row without -inf runs out of
// distinct values before k); then the rounds are done again, one expert at a time.
template <int V, int NV> struct RowTop<float, V, NV> : RowWords<NV> {
    static constexpr bool OWN_ID = false;
    __device__ __forceinline__ int choose(const float (&v)[NV], int k, int lane, int32_t *ids,
                                          uint32_t &key, uint32_t &top)
    {
        uint32_t(&word)[NV] = this->word;
        const uint32_t first = uint32_t(expert_of<V>(0, lane));
        this->last = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            word[i] = order_key(v[i]);
        uint32_t mine = 0u, wins = 0u, last = 0xFFFFFFFFu;  // (above every key)
        int left = 0;
        for (; left < k; ++left) {
            uint32_t best;
            const uint32_t far = this->descend(best);
            if (this->last == 0u || this->last >= last)
                break;
            last = this->last;
            mine = lane >= left ? last : mine;
            wins |= best == far ? 1u << left : 0u;
        }
        int count = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            count += word[i] >= last;
        if (left == 0 || __reduce_add_sync(0xffffffffu, count) == left) {
            if (lane >= left && lane < k)
                ids[lane] = -1;
            while (__any_sync(0xffffffffu, wins != 0u)) {
                const int j = __ffs(wins) - 1;
                const uint32_t want = __shfl_sync(0xffffffffu, mine, j & 31);
                uint32_t e = 0u;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    e = word[i] == want ? uint32_t(expert_of<V>(i, 0)) : e;
                if (wins)
                    ids[j] = int32_t(first + e);
                wins &= wins - 1u;
            }
        } else {
            left = 0;
            int id = -1;
            for (; left < k; ++left) {
                uint32_t best = word[0];
#pragma unroll
                for (int i = 1; i < NV; ++i)
                    best = max(best, word[i]);
                const uint32_t high = __reduce_max_sync(0xffffffffu, best);
                if (high == 0u)
                    break;
                uint32_t lowest = 0xFFFFFFFFu;
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
                    lowest = word[i] == high ? first + uint32_t(expert_of<V>(i, 0)) : lowest;
                const uint32_t e = __reduce_min_sync(0xffffffffu, lowest);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    word[i] = e - first == uint32_t(expert_of<V>(i, 0)) ? 0u : word[i];
                if (lane == left) {
                    mine = high;
                    id = int(e);
                }
            }
            if (lane < k)
                ids[lane] = id;
        }
        key = lane < left ? mine : 0u;
        top = __shfl_sync(0xffffffffu, key, 0);
        return -1;
    }
};

// weights[t][j], ids[t][j] for the k largest logits of row t, largest first, ties to
// the lowest expert.  One warp per token, k rounds of RowTop; lane j keeps choice j.
// Statistics in FP32.  Bound by the integer unit (71% busy at 65521 x 256 with 8 choices): a
// round takes a subtraction and a maximum per register.  That size takes 26.9 us in BF16
// (1.4 TB/s) and 39.2 us in FP32 (1.8 TB/s), whose registers are twice the bytes, 2 us more
// with the softmax over all; 8192 x 128 in FP32 5.8 us (logits from L2 or from HBM alike).
// (A warp per row: half a warp would save nothing, the registers' work being the same.)
// Tried: differences by multiply-adds and maxima of three, 30.5 us in BF16.
template <class T, int V, int NV>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
moe_route_kernel(const T *__restrict__ logits, int64_t rows, int E, int k, int renorm,
                 float *__restrict__ weights, int32_t *__restrict__ ids)
{
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = int64_t(gridDim.x) * ROUTE_WARPS;
    int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
    Row<T, V, NV> next;
    if (t < rows)
        next.load(logits + t * E, E, lane);
    for (; t < rows; t += step) {
        float v[NV];
        next.values(E, lane, v);
        make_usable<T>(v);
        if (t + step < rows)
            next.load(logits + (t + step) * E, E, lane);
        RowTop<T, V, NV> row;
        uint32_t my_key, top_key;
        const int my_id = row.choose(v, k, lane, ids + t * k, my_key, top_key);
        const float top = key_value(top_key);
        const float p = my_key ? exp_neg(key_value(my_key) - top) : 0.0f;
        float s = p;
        if (!renorm) {
            s = 0.0f;
            if (top_key) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    s += exp_neg(v[i] - top);
            }
        }
        const float den = warp_sum(s);
        if (lane < k) {
            weights[t * k + lane] = my_key ? p / den : 0.0f;
            if (row.OWN_ID)
                ids[t * k + lane] = my_id;
        }
    }
}

// dlogits = direct - p * G with G = sum_j w_j dw_j: direct is w_j dw_j at the chosen
// experts, p the softmax over the chosen experts (renorm) or over all; at a chosen
// expert p is its weight, so that the element is w_j (dw_j - G).  Every element of the row
// is written, first the row without its choices, then these.  A choice with an id
// outside [0, E) takes no part.  One warp per token, in FP32, rounded once to the logits'
// type.  The row written, and read for the softmax over all: 65521 x 256 with 8 choices in
// FP32 24.5 us (5.8 TB/s) and 18.1 us renormalized (4.0 TB/s); in BF16 20.4 and 14.3 us, bound
// by issue slots (the exponentials and the row's way through shared memory).  These are with
// logits and gradient in HBM; in L2 24.2, 13.7, 20.1 and 11.2 us.
template <class T, int V, int NV>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
moe_route_bwd_kernel(const float *__restrict__ dweights, const float *__restrict__ weights,
                     const int32_t *__restrict__ ids, const T *__restrict__ logits, int64_t rows,
                     int E, int k, int renorm, T *__restrict__ dlogits)
{
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    // the row is put together in shared memory: single elements stored over it in global
    // memory would cost a sector each
    __shared__ __align__(16) T rows_out[ROUTE_WARPS][NV * 32];
    __shared__ uint8_t lanes_out[ROUTE_WARPS][NV * 32];
    T *out = rows_out[threadIdx.x >> 5];
    uint8_t *out_lane = lanes_out[threadIdx.x >> 5];
    const int64_t step = int64_t(gridDim.x) * ROUTE_WARPS;
    int64_t t = int64_t(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
    // the next row's inputs are under way while a row is worked on
    Row<T, V, NV> next;
    int next_id = -1;
    float next_w = 0.0f, next_dw = 0.0f;
    const auto fetch = [&](int64_t at) {
        if (at >= rows)
            return;
        if (!renorm)
            next.load(logits + at * E, E, lane);
        if (lane < k) {
            next_id = ids[at * k + lane];
            next_w = weights[at * k + lane];
            next_dw = dweights[at * k + lane];
        }
    };
    fetch(t);
    for (; t < rows; t += step) {
        const int id = next_id;
        const float w = next_w, dw = next_dw;
        float d[NV];
        if (!renorm) {
            next.values(E, lane, d);
            make_usable<T>(d);
        }
        fetch(t + step);
        const bool some = id >= 0 && id < E;
        const float total = warp_sum(some ? w * dw : 0.0f);
        float g = w * (dw - total);
        if (renorm) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i] = 0.0f;
        } else {
            // p = w0 exp(l - l0), from the weight and the logit of the first choice
            const int id0 = __shfl_sync(0xffffffffu, some ? id : -1, 0);
            const float w0 = __shfl_sync(0xffffffffu, w, 0);
            float top = 0.0f, c = 0.0f;
            if (id0 >= 0) {
                float mine = d[0];
#pragma unroll
                for (int i = 1; i < NV; ++i)
                    mine = id0 - expert_of<V>(0, lane) == expert_of<V>(i, 0) ? d[i] : mine;
                top = __shfl_sync(0xffffffffu, mine, id0 / V & 31);
                c = -total * w0;
            } else {
                // left out: the softmax anew
                float m = d[0], s = 0.0f;
#pragma unroll
                for (int i = 1; i < NV; ++i)
                    m = fmaxf(m, d[i]);
                const uint32_t key = __reduce_max_sync(0xffffffffu, order_key(m));
                top = key ? key_value(key) : 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    s += exp_neg(d[i] - top);
                s = warp_sum(s);
                c = s > 0.0f ? -total / s : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i] = exp_neg(d[i] - top);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i] *= c;
        }
        __syncwarp();  // the last row has left the buffer
        Row<T, V, NV>::store(out, E, lane, d);
        // An expert named twice (never by the router) collects its choices in their order:
        // the sum of w dw, less p G with p the weights' sum.
        if (some)
            out_lane[id] = uint8_t(lane);
        __syncwarp();
        if (__any_sync(0xffffffffu, some && out_lane[id] != lane)) {
            const uint32_t live = __ballot_sync(0xffffffffu, some);
            const uint32_t same = same_key(uint32_t(id), 32 - __clz(E - 1)) & live;
            float sum = 0.0f;
            for (int j = 0; j < k; ++j) {
                const float gj = __shfl_sync(0xffffffffu, g, j);
                if ((same >> j) & 1u)
                    sum += gj;
            }
            g = sum;
        }
        __syncwarp();  // the row comes first
        if (some)
            out[id] = from_f32<T>(g);
        __syncwarp();
        Row<T, V, NV>::copy(dlogits + t * E, out, E, lane);
    }
}

// ------------------------------------------------------------------------- plan

// The pairs (t, j), in order p = t * k + j, are cut into `chunks` equal runs, one CTA
// each, and each CTA's run into one run per warp, which keeps its ids in registers.
// Counting the ids of every run gives, by prefix sums over warps and chunks, the place at
// which each run's first pair of an expert goes; inside a run a warp ranks 32 pairs at a
// time by matching ids.  All sums are of whole numbers, and a pair's place depends on the
// ids alone.
//
// Bound by latency: the ids, the counts of the other chunks and the stores follow each
// other; with many pairs per SM by the stores to src, a line for each pair.  So up to 2^16
// pairs go to one launch, a cluster of up to 16 CTAs that read each other's counts, and
// more to two launches of up to 64 CTAs, the first of which counts (one / two launches, us:
// 16384 pairs 6.6 / 9.4, 32768 pairs 6.3 / 8.9, 65536 pairs 7.9 / 9.1, 96000 pairs 9.5 / 9.1,
// 131040 pairs 10.8 / 9.1; clusters of 8: 6.6, 7.5 and 11.0 at the first three; 30 pairs take
// 4.5, 524168 pairs over 256 experts 15.2).  Ranking in the counting pass, so that the rows
// need no further votes, gains 0.4 us at 30 pairs and loses 3.9 at 524168, where the votes
// then no longer run under the stores.
constexpr int PLAN_WARPS = 32;
constexpr int PLAN_THREADS = PLAN_WARPS * 32;
constexpr int PLAN_PAIRS = 2048;  // pairs of a chunk, at least
constexpr int PLAN_CHUNKS = 64;
constexpr int PLAN_CLUSTER = 16;  // chunks that one cluster takes, at most
constexpr int PLAN_REGS = 16;     // 32-pair steps of a warp's run, at most
constexpr int PLAN_CLUSTER_PAIRS = 1 << 16;  // pairs that one cluster takes, at most

// (the layout holds at most 2^20 rows, and so pairs)
static_assert(int64_t(PLAN_CHUNKS) * PLAN_WARPS * PLAN_REGS * 32 >= (1 << 20), "runs hold all pairs");

// One warp's run: its ids, -1 outside [0, E) and behind the end.
struct PlanRun {
    int lo, hi;
    int id[PLAN_REGS];
    __device__ __forceinline__ void load(const int32_t *ids, int pairs, int E, int chunk, int chunks,
                                         int warp, int lane)
    {
        const int runs = chunks * PLAN_WARPS, r = chunk * PLAN_WARPS + warp;
        const int len = ((pairs + runs - 1) / runs + 31) / 32 * 32;
        lo = int(min(int64_t(pairs), int64_t(r) * len));
        hi = min(pairs, lo + len);
#pragma unroll
        for (int i = 0; i < PLAN_REGS; ++i) {
            const int p = lo + 32 * i + lane;
            const int v = p < hi ? ids[p] : -1;
            id[i] = v >= 0 && v < E ? v : -1;
        }
    }
    // Adds them to cnt[E] (shared).
    __device__ __forceinline__ void count(int *cnt) const
    {
#pragma unroll
        for (int i = 0; i < PLAN_REGS; ++i)
            if (id[i] >= 0)
                atomicAdd(&cnt[id[i]], 1);
    }
};

__global__ void __launch_bounds__(PLAN_THREADS)
moe_plan_count_kernel(const int32_t *__restrict__ ids, int pairs, int E, int *__restrict__ hist)
{
    extern __shared__ int cnt[];  // [E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS)
        cnt[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    PlanRun run;
    run.load(ids, pairs, E, blockIdx.x, gridDim.x, warp, lane);
    run.count(cnt);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS)
        hist[e * PLAN_CHUNKS + blockIdx.x] = cnt[e];
}

__device__ __forceinline__ int ld_cluster_int(const int *p, int rank)
{
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), uint32_t(rank))) : "memory");
    return v;
}

// CLUSTER: the chunks are the CTAs of one cluster and read each other's counts from shared
// memory; otherwise the counts of all chunks come from moe_plan_count_kernel.
template <bool CLUSTER>
__global__ void __launch_bounds__(PLAN_THREADS)
moe_plan_place_kernel(const int32_t *__restrict__ ids, int pairs, int E,
                      const int *__restrict__ hist, int rows, int32_t *__restrict__ seg,
                      int32_t *__restrict__ row, int32_t *__restrict__ src)
{
    extern __shared__ int sh[];
    int *cnt = sh;                      // [PLAN_WARPS][E]
    int *own = cnt + PLAN_WARPS * E;    // [E] this chunk's pairs of the expert
    int *total = own + E;               // [E] all chunks'
    int *base = total + E;              // [E] those of earlier chunks; then the chunk's first row
    int *first = base + E;              // [E + 1] first block of the expert
    __shared__ int warp_blocks[PLAN_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = blockIdx.x, chunks = gridDim.x;
    const int e = threadIdx.x;  // the expert that this thread sums up, if there is one
    static_assert(PLAN_THREADS >= 1024, "a thread per expert");
    for (int i = threadIdx.x; i < PLAN_WARPS * E; i += PLAN_THREADS)
        cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    PlanRun run;
    run.load(ids, pairs, E, chunk, chunks, warp, lane);
    run.count(cnt + warp * E);
    if (!CLUSTER) {
        // all chunks' counts, one warp per expert
#pragma unroll 4
        for (int x = warp; x < E; x += PLAN_WARPS) {
            const int *h = hist + x * PLAN_CHUNKS;
            int t = 0, b = 0;
#pragma unroll
            for (int i = 0; i < PLAN_CHUNKS / 32; ++i) {
                const int c = i * 32 + lane;
                const int n = c < chunks ? h[c] : 0;
                t += n;
                b += c < chunk ? n : 0;
            }
            t = __reduce_add_sync(0xffffffffu, t);
            b = __reduce_add_sync(0xffffffffu, b);
            if (lane == 0) {
                total[x] = t;
                base[x] = b;
            }
        }
    }
    __syncthreads();
    // counts of each warp's run -> how many pairs of the expert come before it in the chunk
    int all = 0, before = 0;
    if (e < E) {
#pragma unroll 8
        for (int w = 0; w < PLAN_WARPS; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = all;
            all += c;
        }
        own[e] = all;
    }
    if (CLUSTER) {
        cluster_sync();
        if (e < E) {
            int n[PLAN_CLUSTER];
            all = 0;
#pragma unroll
            for (int c = 0; c < PLAN_CLUSTER; ++c)
                n[c] = c < chunks ? ld_cluster_int(own + e, c) : 0;
#pragma unroll
            for (int c = 0; c < PLAN_CLUSTER; ++c) {
                all += n[c];
                before += c < chunk ? n[c] : 0;
            }
            total[e] = all;
        }
    } else if (e < E) {
        all = total[e];
        before = base[e];
    }
    // blocks of each expert, summed over the experts before it
    const int blocks = e < E ? (all + 127) / 128 : 0;
    int sum = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        sum += lane >= o ? up : 0;
    }
    if (lane == 31)
        warp_blocks[warp] = sum;
    __syncthreads();
    sum += __reduce_add_sync(0xffffffffu, lane < warp ? warp_blocks[lane] : 0);
    if (e < E) {
        first[e] = sum - blocks;
        base[e] = (sum - blocks) * 128 + before;
        if (e == E - 1)
            first[E] = sum;
    }
    __syncthreads();
    if (chunk == 0)
        for (int i = threadIdx.x; i <= E; i += PLAN_THREADS)
            seg[i] = first[i];
    int *mine = cnt + warp * E;
#pragma unroll
    for (int i = 0; i < PLAN_REGS; ++i) {
        const int p = run.lo + 32 * i + lane, id = run.id[i];
        if (run.lo + 32 * i >= run.hi)
            break;
        // (-1 has a bit of its own above those of the experts)
        const uint32_t same = same_key(uint32_t(id), 33 - __clz(E - 1));
        int at = 0;
        if (id >= 0)
            at = mine[id] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (id >= 0 && lane == 31 - __clz(same))
            mine[id] = at + 1;
        __syncwarp();
        if (p < run.hi) {
            const int r = id >= 0 ? base[id] + at : -1;
            row[p] = r;
            if (r >= 0)
                src[r] = p;
        }
    }
    // rows that no pair takes: the rest of each expert's last block, and all behind the last
    for (int x = chunk * PLAN_WARPS + warp; x < E; x += chunks * PLAN_WARPS)
        for (int r = first[x] * 128 + total[x] + lane; r < first[x + 1] * 128; r += 32)
            src[r] = -1;
    for (int r = first[E] * 128 + chunk * PLAN_THREADS + threadIdx.x; r < rows;
         r += chunks * PLAN_THREADS)
        src[r] = -1;
    if (CLUSTER)
        cluster_sync();  // no peer reads this CTA's counts any more
}

// ------------------------------------------------------------------- host side

template <class K, class... A>
static cudaError_t launch(K kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                          A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    set_pdl(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
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
                      0, 1, stream, static_cast<const T *>(logits), rows, E, k, int(renorm), weights,
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
                      ROUTE_WARPS * 32, 0, 1, stream, dweights, weights, ids,
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

size_t moe_plan_workspace(int E)
{
    return size_t(PLAN_CHUNKS) * size_t(E) * sizeof(int);
}

cudaError_t launch_moe_plan(const int32_t *ids, int64_t T, int k, int E, int32_t *seg,
                            int32_t *row, int32_t *src, void *workspace, cudaStream_t stream)
{
    const int pairs = int(T * k);
    const bool one = pairs <= PLAN_CLUSTER_PAIRS;  // one cluster
    const size_t count_smem = size_t(E) * sizeof(int);
    const size_t place_smem = ((PLAN_WARPS + 4) * size_t(E) + 1) * sizeof(int);
    static LaunchCache cache;  // CTAs of the largest cluster that the GPU takes
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (cache.get(dev) == 0) {
        constexpr int most_smem = ((PLAN_WARPS + 4) * 1024 + 1) * int(sizeof(int));
        e = cudaFuncSetAttribute(moe_plan_place_kernel<true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(moe_plan_place_kernel<false>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(moe_plan_place_kernel<true>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        cudaLaunchConfig_t q = {};
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = PLAN_CLUSTER;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.gridDim = dim3(PLAN_CLUSTER);
        q.blockDim = dim3(PLAN_THREADS);
        q.dynamicSmemBytes = most_smem;
        q.attrs = qa;
        q.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, moe_plan_place_kernel<true>, &q);
        if (e != cudaSuccess)
            return e;
        cache.set(dev, n > 0 ? PLAN_CLUSTER : 8);  // 8 is portable
    }
    const int64_t wanted = (pairs + PLAN_PAIRS - 1) / PLAN_PAIRS, most = one ? cache.get(dev) : PLAN_CHUNKS;
    const int chunks = int(wanted < most ? wanted : most);
    const int rows = int(moe_plan_rows(T, k, E));
    int *hist = static_cast<int *>(workspace);
    if (one)
        return launch(moe_plan_place_kernel<true>, dim3(chunks), PLAN_THREADS, place_smem, chunks,
                      stream, ids, pairs, E, static_cast<const int *>(hist), rows, seg, row, src);
    e = launch(moe_plan_count_kernel, dim3(chunks), PLAN_THREADS, count_smem, 1, stream, ids, pairs, E,
               hist);
    if (e != cudaSuccess)
        return e;
    return launch(moe_plan_place_kernel<false>, dim3(chunks), PLAN_THREADS, place_smem, 1, stream, ids,
                  pairs, E, static_cast<const int *>(hist), rows, seg, row, src);
}

} // namespace fp8bw
