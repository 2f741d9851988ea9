// What the layers for a few tokens share: the list of the experts that have tokens.
#pragma once

#include "common.cuh"

#include <cuda_bf16.h>

namespace moe {

constexpr int kFewEntries = 1024;   // S * K
constexpr int kFewExperts = 1024;
constexpr int kFewWidth = 16384;    // H, F

// Every CTA makes these lists for itself, in shared memory, from topk_idx: at most
// 1024 entries, 1 to 2 us, where a launch that makes them for all would cost as
// much.  Ranks are those of the entries' order, so all CTAs and launches agree.
struct Routing {
    int16_t *count;   // [E] entries of each expert, then its place among those with tokens
    int16_t *hit;     // [hits] experts with tokens
    int16_t *first;   // [hits + 1] first packed row of each
    int16_t *parts;   // [hits + 1] parts of at most `rows` rows before each
    int16_t *order;   // [rows] the entry of each packed row
    int16_t *place;   // [S K] the row of each entry where parts have `rows` rows each, full
                      // or not; -1 without an expert
    int hits;

    static size_t bytes(int n, int E) { return (size_t)(E + 3 * (n < E ? n : E) + 2 + 2 * n) * 2; }

    __device__ Routing(void *smem, int n, int E)
    {
        const int most = min(n, E);
        count = static_cast<int16_t *>(smem);
        hit = count + E;
        first = hit + most;
        parts = first + most + 1;
        order = parts + most + 1;
        place = order + n;
        hits = 0;
    }
};

template <int THREADS>
__device__ void route(const int32_t *idx, int n, int E, int rows, Routing &r)
{
    constexpr int kWarps = THREADS / 32, kEach = kFewExperts / THREADS;
    __shared__ int s_sum[kWarps], s_hits[kWarps], s_parts[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n <= 32) {
        // A warp does it alone, without a look at every expert, which are listed as
        // they come.
        if (warp == 0) {
            int e = lane < n ? __ldg(idx + lane) : -1;
            if (e < 0 || e >= E) e = -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int count = __popc(same), slot = __popc(same & lanemask_lt());
            const bool leads = e >= 0 && slot == 0;
            const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
            int a = leads ? count : 0, d = leads ? (count + rows - 1) / rows : 0;
            const int mine = a, part = d;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, a, o), w = __shfl_up_sync(0xffffffffu, d, o);
                if (lane >= o) a += u, d += w;
            }
            const int h = __popc(leaders & lanemask_lt()), hits = __popc(leaders);
            const int leader = __ffs(same) - 1;
            const int first = __shfl_sync(0xffffffffu, a - mine, leader);
            const int parts = __shfl_sync(0xffffffffu, d - part, leader);
            if (leads) r.hit[h] = e, r.first[h] = first, r.parts[h] = parts;
            if (e >= 0) r.order[first + slot] = lane;
            if (lane < n) r.place[lane] = e >= 0 ? parts * rows + slot : -1;
            if (lane == 31) r.first[hits] = a, r.parts[hits] = d, s_hits[0] = hits;
        }
        __syncthreads();
        r.hits = s_hits[0];
        return;
    }
    for (int e = tid; e < E; e += THREADS) r.count[e] = 0;
    for (int i = tid; i < n; i += THREADS) {
        const int e = __ldg(idx + i);
        r.place[i] = e >= 0 && e < E ? e : -1;
    }
    __syncthreads();
    if (warp == 0) {
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane, e = i < n ? r.place[i] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int before = e >= 0 ? r.count[e] : 0;
            __syncwarp();
            if (e >= 0) {
                r.place[i] = before + __popc(same & lanemask_lt());
                if ((same & lanemask_lt()) == 0) r.count[e] = before + __popc(same);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // a thread owns kEach neighbouring experts
    int c[kEach], sum = 0, some = 0, part = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = tid * kEach + j;
        c[j] = e < E ? r.count[e] : 0;
        sum += c[j];
        some += c[j] > 0;
        part += (c[j] + rows - 1) / rows;
    }
    int a = sum, b = some, d = part;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, a, o), v = __shfl_up_sync(0xffffffffu, b, o),
                  w = __shfl_up_sync(0xffffffffu, d, o);
        if (lane >= o) a += u, b += v, d += w;
    }
    if (lane == 31) s_sum[warp] = a, s_hits[warp] = b, s_parts[warp] = d;
    __syncthreads();
    a -= sum, b -= some, d -= part;
    r.hits = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) a += s_sum[w], b += s_hits[w], d += s_parts[w];
        r.hits += s_hits[w];
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = tid * kEach + j;
        if (e < E) r.count[e] = b;
        if (c[j] > 0) r.hit[b] = e, r.first[b] = a, r.parts[b] = d, ++b;
        a += c[j];
        d += (c[j] + rows - 1) / rows;
    }
    if (tid == THREADS - 1) r.first[b] = a, r.parts[b] = d;
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
        const int e = __ldg(idx + i);
        if (e >= 0 && e < E) {
            const int h = r.count[e], slot = r.place[i];
            r.order[r.first[h] + slot] = i;
            r.place[i] = r.parts[h] * rows + slot;
        }
    }
    __syncthreads();
}

// The entries' weights, in shared memory.
__device__ __forceinline__ void load_weights(const float *topk_w, int n, float *to)
{
    for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = __ldg(topk_w + i);
}

// out[s, o] = sum over the valid entries of s, in increasing k, for N tokens of which
// the first `count` are stored: y [S K, H] holds the experts' rows by entry.  The
// loads are unconditional, so that 8 N of them are under way: with a condition
// each, or a token at a time, 32 tokens took 30 to 50 us.
constexpr int kFewTokens = 4;
template <int N>
__device__ __forceinline__ void few_combine(const float *y, const float *weights,
                                            const int16_t *place, int K, int H, int o,
                                            const int (&s)[kFewTokens], int count, void *out,
                                            bool f32)
{
    constexpr int kAtOnce = 8;
    float sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += kAtOnce) {
        float v[N][kAtOnce];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                v[j][k] = __ldcg(y + (int64_t)(s[j] * K + min(k0 + k, K - 1)) * H + o);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = s[j] * K + min(k0 + k, K - 1);
                // rows of entries without an expert hold anything
                if (k0 + k < K && place[i] >= 0) sum[j] = fmaf(weights[i], v[j][k], sum[j]);
            }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j >= count) break;
        if (f32) static_cast<float *>(out)[(int64_t)s[j] * H + o] = sum[j];
        else
            static_cast<__nv_bfloat16 *>(out)[(int64_t)s[j] * H + o] = __float2bfloat16_rn(sum[j]);
    }
}

// What a call of moe_expert_layer is about.
struct LayerCall {
    const uint8_t *x;        // bf16 [S, H]
    const int32_t *idx;      // [S, K]
    const float *topk_w;     // [S, K]
    const uint8_t *up, *up_scales, *down, *down_scales;
    uint8_t *out;            // [S, H]
    uint8_t *workspace;
    int S, K, E, H, F;
    bool f32;                // type of out
};

// The layer on MXFP4 weights (csrc/expert_layer_mxfp4.cu).
size_t layer_mxfp4_workspace(int64_t S, int64_t K, int64_t E, int64_t H, int64_t F);
int layer_mxfp4(const LayerCall &c, cudaStream_t stream);

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

} // namespace moe
