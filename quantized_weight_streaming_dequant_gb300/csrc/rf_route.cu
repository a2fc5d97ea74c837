// rf_route.cu -- routing of a chunk of tokens: each token's top-k experts and
// their weights, and the chunk's (token, slot) rows in the order of their
// experts (neurostream, "How it works" 2, for many tokens at once).
//
// pick: a warp per token holds its logits in registers as order-preserving
// integer keys; k rounds of two warp reductions (the largest key, then the
// lowest expert that has it).  place: a stable counting sort by expert.  The
// chunk is cut into at most kBlocks runs of tokens; pick leaves each run's
// counts, and a run's place is the sum of what comes before it (every block
// adds the counts up itself: at most kBlocks * n_expert integers out of L2).
// Within a run, warps take consecutive pieces, and a warp's rows of the same
// expert find their rank with one match.  Up to kOneTokens tokens take one
// launch of one block, more take two launches.
// Bound: chains of dependent steps in two short launches (place: the runs'
// counts, a scan over the experts, ranks by match, each behind a barrier).
// 2.6 MB for 8192 tokens of 128 bf16 logits are 0.4 us of memory time, and the
// two launches take 5 and 7 (4 and 5 with the logits in L2); 5 tokens of 128
// fp32 logits take 3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "rf_chunk.h"
#include "rf_device.cuh"

namespace rf {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBlocks = 128;       // runs of tokens, unless they would be longer than kMaxRun
constexpr int kMaxRun = 65535;     // (a run's counts are 16 bits)
constexpr int kRunTokens = 32;     // tokens per run at least
constexpr int kOneTokens = 64;     // up to here one block does both steps
constexpr int kMaxExperts = 1024;

struct RouteParams {
    const void *logits;
    int64_t ld, n_tok;
    int32_t n_expert, top_k, run, runs;
    int32_t *idx;
    float *w;
    int32_t *offsets, *order, *place;
    int32_t *counts;               // [runs][n_expert]
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Keys order like the logits: NaN counts as -inf, the two zeros are equal.
// 0 is below every key.
__device__ __forceinline__ uint32_t key_of(float v)
{
    if (v != v) v = -INFINITY;
    const uint32_t b = __float_as_uint(v + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

// Tokens [t0, t1), a warp each; counts: the block's counts by expert, or NULL.
template <class T, int EPL>
__device__ __forceinline__ void pick(const RouteParams &p, int64_t t0, int64_t t1, int *counts)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = t0 + warp; t < t1; t += kWarps) {
        const T *x = static_cast<const T *>(p.logits) + t * p.ld;
        uint32_t key[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = lane + 32 * i < p.n_expert ? key_of(as_f32(x[lane + 32 * i])) : 0u;
        float e = 0.f, m = 0.f, sum = 0.f;
        int mine = 0;
        for (int k = 0; k < p.top_k; ++k) {
            uint32_t best = key[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(0xffffffffu, best);
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int i = EPL - 1; i >= 0; --i)
                if (key[i] == best) at = (uint32_t)(lane + 32 * i);
            at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (at == (uint32_t)(lane + 32 * i)) key[i] = 0u;
            const float v = value_of(best);
            if (k == 0) m = v;
            const float ev = expf(v - m);
            sum += ev;
            if (lane == k) e = ev, mine = (int)at;
        }
        if (lane < p.top_k) {
            p.idx[t * p.top_k + lane] = mine;
            p.w[t * p.top_k + lane] = e / sum;
            if (counts) atomicAdd(&counts[mine], 1);
        }
    }
}

template <class T, int EPL>
__global__ void __launch_bounds__(kThreads) pick_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ int counts[kMaxExperts];
    for (int e = threadIdx.x; e < p.n_expert; e += kThreads) counts[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * p.run;
    pick<T, EPL>(p, t0, min(p.n_tok, t0 + p.run), counts);
    __syncthreads();
    for (int e = threadIdx.x; e < p.n_expert; e += kThreads) p.counts[(int64_t)blockIdx.x * p.n_expert + e] = counts[e];
}

// The rows of run `b`, whose idx are written: their places among all rows.
// (own: this block is the only one, and counts its rows itself.)
__device__ __forceinline__ void place_run(const RouteParams &p, int b, bool own)
{
    __shared__ int s_base[kMaxExperts];              // rows before this run's, by expert
    __shared__ uint16_t s_warp[kWarps][kMaxExperts]; // ... and before this warp's, within the run
    __shared__ int s_all[kMaxExperts], s_earlier[kMaxExperts];   // rows of all runs, and of earlier ones, by expert
    __shared__ int s_part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t f0 = (int64_t)b * p.run * p.top_k, f1 = min(p.n_tok, (int64_t)(b + 1) * p.run) * p.top_k;
    const int n = (int)(f1 - f0);
    const int each = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;   // rows per warp
    for (int e = tid; e < p.n_expert; e += kThreads) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_warp[w][e] = 0;   // (each warp's own counts)
        s_all[e] = s_earlier[e] = 0;
    }
    __syncthreads();
    if (!own) {
        // The runs' counts, by expert and share of the runs.
        const int width = (p.n_expert + 31) / 32 * 32, shares = max(1, kThreads / width);
        for (int e = tid % width + (tid / width >= shares ? p.n_expert : 0); e < p.n_expert; e += kThreads) {
            int all = 0, earlier = 0;
#pragma unroll 8
            for (int r = shares > 1 ? tid / width : 0; r < p.runs; r += shares) {
                const int c = p.counts[(int64_t)r * p.n_expert + e];
                all += c;
                if (r < b) earlier += c;
            }
            atomicAdd(&s_all[e], all);
            atomicAdd(&s_earlier[e], earlier);
        }
    }
    // Counts by warp.
    const int from = warp * each, to = min(n, from + each);
    for (int i0 = from; i0 < to; i0 += 32) {
        const int e = i0 + lane < to ? p.idx[f0 + i0 + lane] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) s_warp[warp][e] += (uint16_t)__popc(same);
        __syncwarp();
    }
    __syncthreads();
    // Experts in order, kThreads at a time: rows of earlier experts, and of
    // this expert in earlier runs.
    int before = 0;
    for (int e0 = 0; e0 < p.n_expert; e0 += kThreads) {
        const int e = e0 + tid;
        int all = 0, earlier = 0;
        if (e < p.n_expert) {
            int run = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int c = s_warp[w][e];
                s_warp[w][e] = (uint16_t)run;
                run += c;
            }
            all = own ? run : s_all[e];
            earlier = s_earlier[e];
        }
        int x = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_part[warp] = x;
        __syncthreads();
        int lower = before, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) lower += s_part[w];
            total += s_part[w];
        }
        if (e < p.n_expert) {
            const int start = lower + x - all;
            s_base[e] = start + earlier;
            if (b == 0) {
                p.offsets[e] = start;
                if (e == p.n_expert - 1) p.offsets[e + 1] = start + all;
            }
        }
        before += total;
        __syncthreads();
    }
    // Places, each warp's rows in order.
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < to ? p.idx[f0 + i] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int at = e < 0 ? 0 : s_base[e] + s_warp[warp][e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) s_warp[warp][e] += (uint16_t)__popc(same);
        __syncwarp();
        if (e >= 0) {
            p.order[at] = (int32_t)(f0 + i);
            p.place[f0 + i] = at;
        }
    }
}

__global__ void __launch_bounds__(kThreads) place_kernel(const __grid_constant__ RouteParams p)
{
    place_run(p, (int)blockIdx.x, false);
}

template <class T, int EPL>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteParams p)
{
    pick<T, EPL>(p, 0, p.n_tok, nullptr);
    __syncthreads();   // (idx as this block wrote it)
    place_run(p, 0, true);
}

__global__ void zero_kernel(int32_t *offsets, int n)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) offsets[i] = 0;
}

int run_tokens(int64_t n_tok)
{
    return (int)std::min<int64_t>(kMaxRun, std::max<int64_t>(kRunTokens, (n_tok + kBlocks - 1) / kBlocks));
}

template <class T, int EPL>
rf_status launch_one(const RouteParams &p, cudaStream_t s)
{
    if (p.runs == 1) {
        route_kernel<T, EPL><<<1, kThreads, 0, s>>>(p);
        return last_cuda_error();
    }
    pick_kernel<T, EPL><<<(unsigned)p.runs, kThreads, 0, s>>>(p);
    if (last_cuda_error() != RF_OK) return RF_ERR_CUDA;
    place_kernel<<<(unsigned)p.runs, kThreads, 0, s>>>(p);
    return last_cuda_error();
}
template <class T>
rf_status launch_type(const RouteParams &p, cudaStream_t s)
{
    if (p.n_expert <= 32) return launch_one<T, 1>(p, s);
    if (p.n_expert <= 64) return launch_one<T, 2>(p, s);
    if (p.n_expert <= 128) return launch_one<T, 4>(p, s);
    if (p.n_expert <= 256) return launch_one<T, 8>(p, s);
    return launch_one<T, 32>(p, s);
}

}  // namespace

size_t route_workspace(int64_t n_tok, int n_expert, int top_k)
{
    (void)top_k;
    if (n_tok <= kOneTokens) return 0;
    // As many runs as any chunk of up to n_tok tokens has.
    const int64_t runs = std::min<int64_t>((n_tok + kRunTokens - 1) / kRunTokens, std::max<int64_t>(kBlocks, (n_tok + kMaxRun - 1) / kMaxRun));
    return (size_t)runs * n_expert * sizeof(int32_t);
}

rf_status launch_route_tokens(int dtype, const void *logits, int64_t ld, int64_t n_tok, int n_expert, int top_k,
                              int32_t *idx, float *w, int32_t *offsets, int32_t *order, int32_t *place, void *workspace,
                              cudaStream_t s)
{
    if (n_tok == 0) {
        zero_kernel<<<(n_expert + 256) / 256, 256, 0, s>>>(offsets, n_expert + 1);
        return last_cuda_error();
    }
    RouteParams p;
    p.logits = logits, p.ld = ld, p.n_tok = n_tok;
    p.n_expert = n_expert, p.top_k = top_k;
    p.run = n_tok <= kOneTokens ? (int)n_tok : run_tokens(n_tok);
    p.runs = (int)((n_tok + p.run - 1) / p.run);
    p.idx = idx, p.w = w, p.offsets = offsets, p.order = order, p.place = place;
    p.counts = static_cast<int32_t *>(workspace);
    if (dtype == RF_F32) return launch_type<float>(p, s);
    if (dtype == RF_F16) return launch_type<__half>(p, s);
    return launch_type<__nv_bfloat16>(p, s);
}

}  // namespace rf
