// Gradient of the weighted combine.
//
// The combine computes out[s] = sum_k w[s,k] * y[map[s,k]].  With dout the
// gradient of out,
//   dy[map[s,k], j] = w[s,k] * dout[s,j]
//   dw[s,k]         = sum_j dout[s,j] * y[map[s,k], j]     (0 without a row)
// and dy is zero on the rows that no entry reaches: the ends of padded
// buckets and what lies past the last one.
//
// A CTA owns one token: its dout row is read once for each eight entries and
// serves both products of them, so up to K = 8 the call moves S*H of dout, V*H
// of y and R*H of dy and nothing twice.  A thread takes 16 bytes of y per entry and step, all of a
// step's loads issued before the first product; its K sums stay in registers
// in f32 and the CTA joins them in a fixed order (lanes by shuffles, then
// warps in increasing order), so dw does not depend on timing.
//
// Bound by memory: 4096 tokens, K = 8, H = 7168 in bf16 move 999 MB in 148 us
// (6.74 TB/s; 151 us without the streaming hint on bf16 stores, which costs f32
// rows 2 us), 4096 x 4096 in f32 with 12 % padding 1198 MB in 182 us (6.59
// TB/s).  The block scheduler hands tokens to whichever SM is free.  CTAs of
// 256 threads at these sizes: 158 us (bf16).  With few tokens a CTA takes up to
// 512 threads, to spread a token's row.

#include "common.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kEntries = 8;        // entries of a token held in registers at a time
constexpr int kMaxThreads = 512;
// CTAs that clear the rows without an entry, one for each MB of dy up to one per
// SM.  They come first in the grid: at its end they ran alone, and 75 MB of
// padding in 604 MB of rows cost 197 instead of 182 us (608 of them: 190 us).
constexpr int kMaxGapCtas = 152;

__device__ uint32_t g_backward_error;  // kErrCombineIndex

struct BackwardArgs {
    const uint8_t *dout;     // [S, H]
    const uint8_t *y;        // [rows, H]
    const float *w;          // [S, K]
    const int64_t *map;      // [S, K] row or -1
    const int32_t *cnt;      // [E] rows filled per bucket
    const int64_t *off;      // [E + 1] first rows of the buckets
    int64_t S, H, rows;
    int K, E;
    int gap_ctas;
    uint8_t *dy;             // [rows, H]
    float *dw;               // [S, K]
};

// n elements of T as floats, from 16-byte (or 8-byte) loads
template <typename T, int N> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const uint8_t *p) { v = ld_stream16(p); }
    __device__ __forceinline__ void widen(float (&f)[8]) const
    {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[2 * q] = __uint_as_float(u[q] << 16);
            f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void store(uint8_t *p, const float (&f)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
            u[q] = *reinterpret_cast<uint32_t *>(&b);
        }
        st16_cs(p, make_uint4(u[0], u[1], u[2], u[3]));
    }
};
template <> struct Vec<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const uint8_t *p) { v = ld_stream8(p); }
    __device__ __forceinline__ void widen(float (&f)[4]) const
    {
        f[0] = __uint_as_float(v.x << 16);
        f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16);
        f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <> struct Vec<float, 4> {
    uint4 v;
    __device__ __forceinline__ void load(const uint8_t *p) { v = ld_stream16(p); }
    __device__ __forceinline__ void widen(float (&f)[4]) const
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static void store(uint8_t *p, const float (&f)[4])
    {
        st16(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3])));
    }
};
template <> struct Vec<float, 8> {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint8_t *p)
    {
        a = ld_stream16(p);
        b = ld_stream16(p + 16);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const
    {
        f[0] = __uint_as_float(a.x);
        f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z);
        f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x);
        f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z);
        f[7] = __uint_as_float(b.w);
    }
};

template <typename Td, typename Ty>
__global__ void __launch_bounds__(kMaxThreads) combine_backward_kernel(BackwardArgs a)
{
    griddep_wait();  // every input comes from earlier stream work
    griddep_launch_dependents();

    constexpr int N = 16 / (int)sizeof(Ty);  // elements per step
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int64_t row_bytes = a.H * (int)sizeof(Ty);

    if ((int)blockIdx.x < a.gap_ctas) {
        zero_gaps(a.dy, row_bytes, a.rows, a.cnt, a.off, a.E, (int)blockIdx.x * warps + warp,
                  a.gap_ctas * warps);
        return;
    }

    __shared__ int64_t s_at[kEntries];
    __shared__ float s_w[kEntries];
    __shared__ float s_part[kMaxThreads / 32][kEntries];
    const int64_t s = (int64_t)blockIdx.x - a.gap_ctas;
    const uint8_t *dout = a.dout + s * a.H * (int)sizeof(Td);
    const int steps = (int)(a.H / N);

    for (int k0 = 0; k0 < a.K; k0 += kEntries) {
        if (k0) __syncthreads();  // the shared arrays of the entries before
        if (tid < kEntries) {
            int64_t r = -1;
            float w = 0.0f;
            if (k0 + tid < a.K) {
                r = a.map[s * a.K + k0 + tid];
                w = a.w[s * a.K + k0 + tid];
                if (r < -1 || r >= a.rows) {
                    atomicOr(&g_backward_error, kErrCombineIndex);  // dropped, never touched
                    r = -1;
                }
            }
            s_at[tid] = r < 0 ? -1 : r * row_bytes;
            s_w[tid] = w;
        }
        __syncthreads();
        float acc[kEntries];
#pragma unroll
        for (int k = 0; k < kEntries; ++k) acc[k] = 0.0f;
        for (int p = tid; p < steps; p += blockDim.x) {
            Vec<Ty, N> v[kEntries];
            Vec<Td, N> d;
            d.load(dout + (int64_t)p * N * (int)sizeof(Td));
#pragma unroll
            for (int k = 0; k < kEntries; ++k)
                if (s_at[k] >= 0) v[k].load(a.y + s_at[k] + (int64_t)p * 16);
            float fd[N];
            d.widen(fd);
#pragma unroll
            for (int k = 0; k < kEntries; ++k) {
                if (s_at[k] < 0) continue;
                float f[N], g[N];
                v[k].widen(f);
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    acc[k] = fmaf(fd[q], f[q], acc[k]);
                    g[q] = s_w[k] * fd[q];
                }
                Vec<Ty, N>::store(a.dy + s_at[k] + (int64_t)p * 16, g);
            }
        }
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
            if (lane == 0) s_part[warp][k] = acc[k];
        }
        __syncthreads();
        if (tid < kEntries && k0 + tid < a.K) {
            float sum = 0.0f;
            for (int i = 0; i < warps; ++i) sum += s_part[i][tid];
            a.dw[s * a.K + k0 + tid] = sum;
        }
    }
}

template <typename Td, typename Ty>
int launch_backward(const BackwardArgs &a, cudaStream_t stream)
{
    const int steps = (int)(a.H / (16 / (int)sizeof(Ty)));
    int threads = 128;
    while (threads < kMaxThreads && threads < steps && a.S * threads < (int64_t)sm_count() * 1024)
        threads *= 2;
    cudaError_t e = launch_pdl(combine_backward_kernel<Td, Ty>, dim3((unsigned)(a.S + a.gap_ctas)),
                               dim3(threads), 0, stream, a);
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT int moe_combine_backward(const void *dout, int dout_dtype, const void *y,
                                    int64_t y_rows, int y_dtype, const float *topk_w,
                                    const int64_t *tok_map, const int32_t *cnt,
                                    const int64_t *off, int64_t S, int64_t H, int K, int E,
                                    void *dy, float *dw, moe_stream_t stream)
{
    MOE_TRACE("moe_combine_backward");
    if ((dout_dtype != MOE_BF16 && dout_dtype != MOE_F32) ||
        (y_dtype != MOE_BF16 && y_dtype != MOE_F32))
        return MOE_EINVAL;
    if (S < 0 || H < 1 || K < 1 || K > 32 || E < 1 || E > 1024) return MOE_EINVAL;
    if (S >= ((int64_t)1 << 31) / K || H >= ((int64_t)1 << 31)) return MOE_EINVAL;
    if (S + kMaxGapCtas >= ((int64_t)1 << 31)) return MOE_EINVAL;  // CTAs of a grid
    if (S == 0 && y_rows == 0) return MOE_OK;  // no token and no row to clear
    if (y_rows < 1 || y_rows >= ((int64_t)1 << 31) || !dy || !cnt || !off) return MOE_EINVAL;
    if (S > 0 && (!dout || !y || !topk_w || !tok_map || !dw)) return MOE_EINVAL;
    if (H % 8 || !aligned16(dout) || !aligned16(y) || !aligned16(dy)) return MOE_EALIGN;
    BackwardArgs a = {};
    a.dout = static_cast<const uint8_t *>(dout);
    a.y = static_cast<const uint8_t *>(y);
    a.w = topk_w;
    a.map = tok_map;
    a.cnt = cnt;
    a.off = off;
    a.S = S;
    a.H = H;
    a.rows = y_rows;
    a.K = K;
    a.E = E;
    a.dy = static_cast<uint8_t *>(dy);
    a.dw = dw;
    const int64_t mb = (y_rows * H * (y_dtype == MOE_BF16 ? 2 : 4) >> 20) + 1;
    a.gap_ctas = (int)(mb < kMaxGapCtas ? mb : kMaxGapCtas);
    cudaStream_t st = (cudaStream_t)stream;
    if (y_dtype == MOE_BF16)
        return dout_dtype == MOE_BF16 ? launch_backward<__nv_bfloat16, __nv_bfloat16>(a, st)
                                      : launch_backward<float, __nv_bfloat16>(a, st);
    return dout_dtype == MOE_BF16 ? launch_backward<__nv_bfloat16, float>(a, st)
                                  : launch_backward<float, float>(a, st);
}

namespace moe {
// Reads and clears this file's device error bits.
cudaError_t read_backward_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_backward_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_backward_error, &zero, sizeof(uint32_t));
    return e;
}
} // namespace moe
