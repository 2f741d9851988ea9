// Global L2 norm of many gradients, and the gradients scaled to a limit.
//
//   norm = sqrt(sum over all tensors of g^2)
//   c    = min(1, max_norm / (norm + 1e-6)), 1 without a limit (infinity)
//   out  = c * g, rounded once to the tensor's type
//
// The norm has to be known before the first product, so the data is passed
// over twice: one launch sums squares, one scales.  Both walk the same chunks
// (32 KB of one tensor each); the tensors' addresses, sizes and first chunks
// travel in the kernel's parameters, so any mix of sizes is one launch and
// nothing is copied to the device first.  Squares are summed in f32 in a fixed
// tree: four sums a thread, then lanes, warps and CTAs (one partial sum each,
// which every CTA of the second launch adds in the same order).  All terms are
// positive and the longest chain is a few hundred additions at 4 GB, so the
// norm is off by about 1e-7 of itself; f64 sums of the partials would cost the
// second launch 110 us there (this part adds few f64 values a cycle).  The
// result does not depend on timing and no CTA waits for another.  The second
// pass walks the chunks backwards, so that what the first pass read last is
// still in L2.

#include "common.cuh"

#include <cuda_bf16.h>
#include <math.h>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 32768;   // of a gradient, per CTA and step
// CTAs of a launch, and partial sums of one call: four waves of 8 CTAs on 152
// SMs.  SMs of this part do not move data at the same rate, so one wave waits
// for the slowest: 4.54 GB of f32 gradients take 625 us for the norm (7.27
// TB/s) and 1976 us for norm and clipping, against 741 and 2164 us in one.
constexpr int kMaxPartials = 4 * 1216;
constexpr float kEps = 1e-6f;

// The tensors of one launch, passed by value.  Two sizes: a short parameter
// block costs the launch less.
template <int N> struct Table {
    const uint8_t *in[N];
    uint8_t *out[N];
    int64_t numel[N];
    int64_t first[N];    // first chunk
    uint8_t f32[N];
    int64_t chunks;
    int n;
    bool in_place;       // every output is its input
};
constexpr int kShort = 64, kLong = 512;

struct Chunk {
    const uint8_t *in;
    uint8_t *out;
    int n;          // elements
    bool f32;
};

template <int N> __device__ __forceinline__ Chunk chunk_of(const Table<N> &t, int64_t c)
{
    int lo = 0, hi = t.n - 1;  // the last tensor whose first chunk is at or before c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    Chunk r;
    r.f32 = t.f32[lo] != 0;
    const int size = r.f32 ? 4 : 2, per = kChunkBytes / size;
    const int64_t at = (c - t.first[lo]) * per;
    r.n = (int)min((int64_t)per, t.numel[lo] - at);
    r.in = t.in[lo] + at * size;
    r.out = t.out[lo] ? t.out[lo] + at * size : nullptr;
    return r;
}

__device__ __forceinline__ float bf16_at(const uint8_t *p, int i)
{
    return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
}

__device__ __forceinline__ float square4(uint4 v, bool f32, float s)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (f32) {
            const float f = __uint_as_float(u[q]);
            s = fmaf(f, f, s);
        } else {
            const float a = __uint_as_float(u[q] << 16), b = __uint_as_float(u[q] & 0xffff0000u);
            s = fmaf(a, a, s);
            s = fmaf(b, b, s);
        }
    }
    return s;
}

__device__ __forceinline__ uint4 scale4(uint4 v, bool f32, float c)
{
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (f32) {
            u[q] = __float_as_uint(__uint_as_float(u[q]) * c);
        } else {
            __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(u[q] << 16) * c,
                                                     __uint_as_float(u[q] & 0xffff0000u) * c);
            u[q] = *reinterpret_cast<uint32_t *>(&b);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float scalar_at(const Chunk &k, int i)
{
    return k.f32 ? reinterpret_cast<const float *>(k.in)[i] : bf16_at(k.in, i);
}

__device__ __forceinline__ void scalar_put(const Chunk &k, int i, float f)
{
    if (k.f32) reinterpret_cast<float *>(k.out)[i] = f;
    else reinterpret_cast<__nv_bfloat16 *>(k.out)[i] = __float2bfloat16_rn(f);
}

// Elements of the chunk before its first 16-byte boundary, and 16-byte groups.
__device__ __forceinline__ void split(const Chunk &k, int &head, int &groups)
{
    const int size = k.f32 ? 4 : 2;
    head = min(k.n, (int)((16 - (reinterpret_cast<uintptr_t>(k.in) & 15)) & 15) / size);
    groups = (k.n - head) / (16 / size);
}

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float s_warp[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += s_warp[i];
    return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<N> t,
                                                           float *partial)
{
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    float s[4] = {};
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Chunk k = chunk_of(t, c);
        int head, groups;
        split(k, head, groups);
        const int size = k.f32 ? 4 : 2;
        const uint8_t *body = k.in + head * size;
        int i = tid;
        for (; i + 3 * kThreads < groups; i += 4 * kThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ld_stream16(body + (int64_t)(i + j * kThreads) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = square4(v[j], k.f32, s[j]);
        }
        for (; i < groups; i += kThreads)
            s[0] = square4(ld_stream16(body + (int64_t)i * 16), k.f32, s[0]);
        const int done = head + groups * (16 / size);
        if (tid < head) {
            const float f = scalar_at(k, tid);
            s[1] = fmaf(f, f, s[1]);
        }
        if (done + tid < k.n) {
            const float f = scalar_at(k, done + tid);
            s[2] = fmaf(f, f, s[2]);
        }
    }
    const float sum = block_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (tid == 0) partial[blockIdx.x] = sum;
}

// Adds the partial sums, writes the norm (the CTA 0 of the first launch) and
// scales.  max_norm < 0: the norm alone.
template <int N>
__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ Table<N> t, const float *partial, int n_partial,
             float max_norm, float *norm_out)
{
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    float v = 0.0f;
    for (int i = tid; i < n_partial; i += kThreads) v += partial[i];
    const float norm = sqrtf(block_sum(v));
    if (norm_out && blockIdx.x == 0 && tid == 0) *norm_out = norm;
    if (max_norm < 0.0f) return;
    float c = max_norm / (norm + kEps);
    if (c > 1.0f || isinf(max_norm)) c = 1.0f;  // a NaN stays under a finite limit
    if (c == 1.0f && t.in_place) return;  // the values are already there
    for (int64_t b = blockIdx.x; b < t.chunks; b += gridDim.x) {
        const Chunk k = chunk_of(t, t.chunks - 1 - b);
        const int size = k.f32 ? 4 : 2;
        if ((reinterpret_cast<uintptr_t>(k.in) ^ reinterpret_cast<uintptr_t>(k.out)) & 15) {
            // input and output start at different places of a 16-byte group
            for (int i = tid; i < k.n; i += kThreads) scalar_put(k, i, scalar_at(k, i) * c);
            continue;
        }
        int head, groups;
        split(k, head, groups);
        const uint8_t *from = k.in + head * size;
        uint8_t *to = k.out + head * size;
        int i = tid;
        for (; i + 3 * kThreads < groups; i += 4 * kThreads) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = *reinterpret_cast<const uint4 *>(from + (int64_t)(i + j * kThreads) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st16_cs(to + (int64_t)(i + j * kThreads) * 16, scale4(x[j], k.f32, c));
        }
        for (; i < groups; i += kThreads)
            st16_cs(to + (int64_t)i * 16,
                    scale4(*reinterpret_cast<const uint4 *>(from + (int64_t)i * 16), k.f32, c));
        const int done = head + groups * (16 / size);
        if (tid < head) scalar_put(k, tid, scalar_at(k, tid) * c);
        if (done + tid < k.n) scalar_put(k, done + tid, scalar_at(k, done + tid) * c);
    }
}

// Tensors [i0, n) that fit one table; returns the first one left over.
template <int N>
int fill(Table<N> &t, const void *const *in, void *const *out, const int64_t *numel,
         const int *dtype, int i0, int n)
{
    t.n = 0;
    t.chunks = 0;
    t.in_place = true;
    int i = i0;
    for (; i < n && t.n < N; ++i) {
        if (numel[i] == 0) continue;
        const bool f32 = dtype[i] == MOE_F32;
        t.in[t.n] = static_cast<const uint8_t *>(in[i]);
        t.out[t.n] = out ? static_cast<uint8_t *>(out[i]) : nullptr;
        t.in_place = t.in_place && t.out[t.n] == t.in[t.n];
        t.numel[t.n] = numel[i];
        t.first[t.n] = t.chunks;
        t.f32[t.n] = f32;
        const int64_t per = kChunkBytes / (f32 ? 4 : 2);
        t.chunks += (numel[i] + per - 1) / per;
        ++t.n;
    }
    return i;
}

template <int N>
int run(const void *const *in, void *const *out, const int64_t *numel, const int *dtype, int n,
        float max_norm, float *norm, float *partial, cudaStream_t stream)
{
    const int launches = n <= N ? 1 : (n + N - 1) / N;
    const int per = kMaxPartials / launches > 0 ? kMaxPartials / launches : 1;
    Table<N> t;
    int used = 0;
    cudaError_t e = cudaSuccess;
    for (int i = 0, l = 0; l < launches && e == cudaSuccess; ++l) {
        i = fill(t, in, nullptr, numel, dtype, i, n);
        const int grid = (int)(t.chunks < per ? t.chunks : per);
        if (grid == 0) continue;
        e = launch_pdl(squares_kernel<N>, dim3(grid), dim3(kThreads), 0, stream, t, partial + used);
        used += grid;
    }
    for (int i = 0, l = 0; l < launches && e == cudaSuccess; ++l) {
        i = fill(t, in, out, numel, dtype, i, n);
        int grid = out ? (int)(t.chunks < kMaxPartials ? t.chunks : kMaxPartials) : 1;
        if (grid == 0) {
            if (l > 0) continue;
            grid = 1;  // the norm of nothing
        }
        e = launch_pdl(scale_kernel<N>, dim3(grid), dim3(kThreads), 0, stream, t,
                       (const float *)partial, used, max_norm, l == 0 ? norm : nullptr);
        if (!out) break;
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

int check_and_run(const void *const *in, void *const *out, const int64_t *numel, const int *dtype,
                  int n, float max_norm, float *norm, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream)
{
    if (n < 0 || n > MOE_GRAD_TENSORS_MAX || !norm) return MOE_EINVAL;
    if (n > 0 && (!in || !numel || !dtype)) return MOE_EINVAL;
    if (!workspace || workspace_bytes < moe_grad_norm_workspace_size()) return MOE_EINVAL;
    for (int i = 0; i < n; ++i) {
        if (dtype[i] != MOE_BF16 && dtype[i] != MOE_F32) return MOE_EINVAL;
        if (numel[i] < 0 || numel[i] > ((int64_t)1 << 46)) return MOE_EINVAL;
        if (numel[i] > 0 && (!in[i] || (out && !out[i]))) return MOE_EINVAL;
    }
    const uintptr_t ws = reinterpret_cast<uintptr_t>(workspace);
    if (ws & 255 || reinterpret_cast<uintptr_t>(norm) & 3) return MOE_EALIGN;
    for (int i = 0; i < n; ++i) {
        const uintptr_t mask = dtype[i] == MOE_F32 ? 3 : 1;
        if (numel[i] > 0 && ((reinterpret_cast<uintptr_t>(in[i]) & mask) ||
                             (out && (reinterpret_cast<uintptr_t>(out[i]) & mask))))
            return MOE_EALIGN;
    }
    float *partial = static_cast<float *>(workspace);
    return n <= kShort ? run<kShort>(in, out, numel, dtype, n, max_norm, norm, partial, stream)
                       : run<kLong>(in, out, numel, dtype, n, max_norm, norm, partial, stream);
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT size_t moe_grad_norm_workspace_size(void)
{
    return (kMaxPartials * sizeof(float) + 255) / 256 * 256;
}

MOE_EXPORT int moe_grad_norm(const void *const *grads, const int64_t *numel, const int *dtype,
                             int n, float *norm, void *workspace, size_t workspace_bytes,
                             moe_stream_t stream)
{
    MOE_TRACE("moe_grad_norm");
    return check_and_run(grads, nullptr, numel, dtype, n, -1.0f, norm, workspace, workspace_bytes,
                         (cudaStream_t)stream);
}

MOE_EXPORT int moe_clip_grad_norm(const void *const *grads, void *const *out,
                                  const int64_t *numel, const int *dtype, int n, float max_norm,
                                  float *norm, void *workspace, size_t workspace_bytes,
                                  moe_stream_t stream)
{
    MOE_TRACE("moe_clip_grad_norm");
    if (!(max_norm >= 0.0f) || (n > 0 && !out)) return MOE_EINVAL;
    return check_and_run(grads, out, numel, dtype, n, max_norm, norm, workspace, workspace_bytes,
                         (cudaStream_t)stream);
}
