// MXFP4 rows and weights: quantisation, also on the way into the experts'
// buckets and behind a gated activation, and back to values.
//
// The OCP Microscaling format v1.0 with E2M1 elements: 32 elements of a row
// share a scale 2^(s - 127), s one byte (E8M0, 255 is NaN).  With a the largest
// magnitude of a block, s = floor(log2 a) - 2 + 127, clamped at 0 (so that the
// largest element lands in 4 .. 8, where E2M1 ends at 6), and each code is
// v / 2^(s - 127) rounded to nearest even, saturating at 6.  The division is by a power
// of two and exact wherever the quotient rounds to anything but zero, so the
// codes are a pure function of the values.  A block with an infinite or NaN
// element gets s = 255 and codes of zero: all of it reads back as NaN.
//
// Layout of a [rows, D] tensor: codes [rows, D / 2], element 2i in the low half
// of byte i; scales [ceil(D / 128)][rows][4], the four blocks of 128 elements in
// one word and the words of neighbouring rows side by side, as the experts'
// product copies them (csrc/expert_gemm_mxfp4.cu).  Blocks past D are zero.
//
// A warp takes 512 elements of a row: 16 a lane, two lanes a block, 8 bytes of
// codes a lane, and every eighth lane a word of scales.  A row that goes to K
// buckets is read and rounded once and stored K times.
//
// Bound by memory: 4096 x 7168 bf16 rows into 8 buckets each 34 us (5.4 TB/s of reads and
// scattered rows of codes), their values as bf16 92 us (6.4 TB/s, stores of whole lines;
// 115 us with 32 bytes a lane), 180 M f32 weights 127 us (6.4 TB/s), the activation of
// 32768 x 4096 47.6 us (6.4 TB/s; f32 78 us, 7.3 TB/s).  With 64-bit divisions for each
// unit instead of the walk the dispatch took 37, the weights 132 and the activation 59 us.

#include "common.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLane = 16;             // elements of a lane
constexpr int kUnit = 32 * kLane;     // of a warp
constexpr int kWaves = 8;             // resident waves of the largest grid

__device__ uint32_t g_mxfp4_error;  // kErrDispatchIndex

struct QuantArgs {
    const uint8_t *x;       // [S, D], gated [S, 2 D]
    const int64_t *map;     // [S, K] destination rows, or null: row s to row s
    int64_t S, D;
    int64_t rows;           // destination rows
    int64_t group;          // rows that share a scale array
    int K;
    uint8_t *codes;         // [rows, D / 2]
    uint32_t *scales;       // [rows / group][ceil(D / 128)][group]
};

template <typename T> struct Sixteen;
template <> struct Sixteen<float> {
    __device__ __forceinline__ static void load(const uint8_t *p, float (&f)[kLane])
    {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = ld_stream16(p + 16 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[4 * q] = __uint_as_float(v[q].x);
            f[4 * q + 1] = __uint_as_float(v[q].y);
            f[4 * q + 2] = __uint_as_float(v[q].z);
            f[4 * q + 3] = __uint_as_float(v[q].w);
        }
    }
};
template <> struct Sixteen<__nv_bfloat16> {
    __device__ __forceinline__ static void load(const uint8_t *p, float (&f)[kLane])
    {
        const uint4 v[2] = {ld_stream16(p), ld_stream16(p + 16)};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[8 * q + 2 * i] = __uint_as_float(u[i] << 16);
                f[8 * q + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    }
};

// Four pairs of values as eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float *f)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// h of gates below kFarGate: the fast division gives 0 for divisors above 2^126, which
// 1 + exp(-gate) is below -87.3.  The gates are read again, one by one: they are rare, and kept
// until here they would cost all others registers.  (32768 x 2048 bf16: 47.6 us with and
// without; with the exponential in halves for every gate 52 us.)
template <typename T>
__device__ __forceinline__ void far_gates(const T *gates, uint32_t F, float (&h)[kLane])
{
#pragma unroll 1
    for (int i = 0; i < kLane; ++i) {
        const float gate = (float)gates[i];
        if (!(gate < kFarGate)) continue;
        const float v = far_gate(gate, (float)gates[F + i]);
#pragma unroll
        for (int k = 0; k < kLane; ++k)
            if (k == i) h[k] = v;
    }
}

// A walk over (row, chunk) by all warps of the grid, without a division in it.
struct Walk {
    uint32_t row, chunk, chunks, rows_on, chunks_on;
    __device__ __forceinline__ explicit Walk(uint32_t n) : chunks(n)
    {
        const uint32_t first = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        const uint32_t all = gridDim.x * (kThreads / 32);
        row = first / n;
        chunk = first - row * n;
        rows_on = all / n;
        chunks_on = all - rows_on * n;
    }
    __device__ __forceinline__ void next()
    {
        row += rows_on;
        chunk += chunks_on;
        if (chunk >= chunks) {
            chunk -= chunks;
            ++row;
        }
    }
};

template <typename T, bool GATED, bool MAP>
__global__ void __launch_bounds__(kThreads) quant_kernel(QuantArgs a)
{
    const int lane = threadIdx.x & 31;
    const uint32_t D = (uint32_t)a.D, words = (D + 127) / 128, S = (uint32_t)a.S;
    const uint32_t rows = (uint32_t)a.rows, group = (uint32_t)a.group;
    griddep_wait();
    griddep_launch_dependents();
    for (Walk at((D + kUnit - 1) / kUnit); at.row < S; at.next()) {
        const uint32_t s = at.row, e0 = at.chunk * kUnit + lane * kLane;  // this lane's elements
        const bool in = e0 < D;                     // D is a multiple of two lanes
        int64_t mine = -1;
        if (MAP && lane < a.K) mine = __ldg(a.map + (int64_t)s * a.K + lane);
        float f[kLane];
#pragma unroll
        for (int i = 0; i < kLane; ++i) f[i] = 0.0f;
        if (in) {
            const uint8_t *p = a.x + ((int64_t)s * (GATED ? 2 * D : D) + e0) * (int)sizeof(T);
            Sixteen<T>::load(p, f);
            if (GATED) {
                // f32 with the fast exponential and division: a few units in the last
                // place of 24 bits (2^-16 at a gate of -80), where the codes that
                // follow keep two bits
                float up[kLane], low = 0.0f;
                Sixteen<T>::load(p + (int64_t)D * (int)sizeof(T), up);
#pragma unroll
                for (int i = 0; i < kLane; ++i) {
                    low = fminf(low, f[i]);
                    f[i] = __fdividef(f[i], 1.0f + __expf(-f[i])) * up[i];
                }
                if (low < kFarGate) far_gates(reinterpret_cast<const T *>(p), D, f);
            }
        }
        float most = 0.0f;  // of the magnitudes; NaN if one is
#pragma unroll
        for (int i = 0; i < kLane; i += 2)
            asm("max.NaN.f32 %0, %1, %2, %3;"
                : "=f"(most)
                : "f"(most), "f"(fabsf(f[i])), "f"(fabsf(f[i + 1])));
        uint32_t top = __float_as_uint(most);  // patterns of magnitudes: a NaN's is above all
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const int e = (int)(top >> 23);
        const uint32_t byte = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
        const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);  // 2^(127 - byte)
#pragma unroll
        for (int i = 0; i < kLane; ++i) f[i] *= inv;
        uint2 code = make_uint2(e2m1x8(f), e2m1x8(f + 8));
        if (byte == 255) code = make_uint2(0, 0);
        uint32_t word = byte;
        word |= __shfl_down_sync(0xffffffffu, word, 2) << 8;
        word = (word & 0xffffu) | __shfl_down_sync(0xffffffffu, word, 4) << 16;
        const uint32_t w = at.chunk * 4 + (lane >> 3);
        const bool holds = (lane & 7) == 0 && w < words;
        uint8_t *codes = a.codes + e0 / 2;
        uint32_t *scales = a.scales + (int64_t)w * group;
        if (MAP) {
            // the entries' rows that can be stored, one after another
            const bool fits = mine >= 0 && mine < rows;
            if (!fits && mine != -1) atomicOr(&g_mxfp4_error, kErrDispatchIndex);
            for (uint32_t left = __ballot_sync(0xffffffffu, fits); left; left &= left - 1) {
                const uint32_t r = __shfl_sync(0xffffffffu, (uint32_t)mine, __ffs(left) - 1);
                if (in) st8(codes + (int64_t)r * (D / 2), code);
                if (holds) scales[r] = word;
            }
        } else {
            if (in) st8(codes + (int64_t)s * (D / 2), code);
            const uint32_t g = s / group;
            if (holds) scales[(int64_t)g * words * group + (s - g * group)] = word;
        }
    }
}

struct DequantArgs {
    const uint8_t *codes;
    const uint32_t *scales;
    int64_t rows, D, group;
    uint8_t *out;  // [rows, D]
};

// 16 bytes of values a lane and step, so that a warp's stores are whole lines; `kSteps`
// of them at a time.
template <typename T> struct Dequant {
    static constexpr int kEach = 16 / (int)sizeof(T);   // elements of a lane
    static constexpr int kSteps = 4;
    static constexpr int kUnit = 32 * kEach * kSteps;
};

template <typename T> __global__ void __launch_bounds__(kThreads) dequant_kernel(DequantArgs a)
{
    using Dq = Dequant<T>;
    const int lane = threadIdx.x & 31;
    const uint32_t D = (uint32_t)a.D, words = (D + 127) / 128, rows = (uint32_t)a.rows;
    const uint32_t group = (uint32_t)a.group;
    griddep_wait();
    griddep_launch_dependents();
    for (Walk at((D + Dq::kUnit - 1) / Dq::kUnit); at.row < rows; at.next()) {
        const uint32_t r = at.row, g = r / group;
        const uint8_t *codes = a.codes + (int64_t)r * (D / 2);
        const uint32_t *scales = a.scales + (int64_t)g * words * group + (r - g * group);
        uint8_t *out = a.out + (int64_t)r * D * (int)sizeof(T);
        uint32_t code[Dq::kSteps], word[Dq::kSteps];
#pragma unroll
        for (int k = 0; k < Dq::kSteps; ++k) {
            const uint32_t e = at.chunk * Dq::kUnit + (k * 32 + lane) * Dq::kEach;
            code[k] = word[k] = 0;
            if (e < D) {
                code[k] = Dq::kEach == 8 ? __ldg(reinterpret_cast<const uint32_t *>(codes + e / 2))
                                         : __ldg(reinterpret_cast<const uint16_t *>(codes + e / 2));
                word[k] = __ldg(scales + (int64_t)(e / 128) * group);
            }
        }
#pragma unroll
        for (int k = 0; k < Dq::kSteps; ++k) {
            const uint32_t e = at.chunk * Dq::kUnit + (k * 32 + lane) * Dq::kEach;
            if (e >= D) break;
            const uint32_t byte = word[k] >> (e / 32 % 4 * 8) & 255u;
            const float scale = __uint_as_float(byte == 255 ? 0x7fffffffu
                                                : byte     ? byte << 23
                                                           : 0x00400000u);
            float f[Dq::kEach];
#pragma unroll
            for (int i = 0; i < Dq::kEach; ++i) {
                // the code's exponent and mantissa as those of an f32: 2^-126 of its
                // value, subnormal where it is
                const uint32_t nibble = code[k] >> (4 * i);
                f[i] = __uint_as_float((nibble & 7u) << 22 | (nibble & 8u) << 28) * 0x1p126f * scale;
            }
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sizeof(T) == 4) {
                    u[i] = __float_as_uint(f[i]);
                } else {
                    const __nv_bfloat162 b =
                        __floats2bfloat162_rn(f[2 * i % Dq::kEach], f[(2 * i + 1) % Dq::kEach]);
                    u[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
            }
            st16_cs(out + (int64_t)e * (int)sizeof(T), make_uint4(u[0], u[1], u[2], u[3]));
        }
    }
}

template <auto KERNEL, typename Args>
int launch_units(const Args &a, int64_t units, cudaStream_t stream)
{
    static KernelCache kc;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(KERNEL, 0, kThreads, kc, &per_sm);
    if (e == cudaSuccess) {
        const int64_t warps = kThreads / 32, most = (int64_t)sm_count() * per_sm * kWaves;
        const int64_t grid = (units + warps - 1) / warps;
        e = launch_pdl(KERNEL, dim3((unsigned)(grid < most ? grid : most)), dim3(kThreads), 0,
                       stream, a);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

int64_t units_of(int64_t rows, int64_t D, int unit) { return rows * ((D + unit - 1) / unit); }

constexpr int64_t kMaxWidth = 1 << 24;

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What all of these calls ask of a tensor of `groups` [rows, D].
int check_tensor(int64_t groups, int64_t rows, int64_t D)
{
    if (groups < 0 || rows < 0 || D < 1 || D >= kMaxWidth) return MOE_EINVAL;
    if (groups > 0 && rows >= ((int64_t)1 << 31) / groups) return MOE_EINVAL;
    return MOE_OK;
}

template <bool GATED, bool MAP> int run_quant(const QuantArgs &a, int dtype, cudaStream_t stream)
{
    const int64_t units = units_of(a.S, a.D, kUnit);
    if (dtype == MOE_F32) return launch_units<quant_kernel<float, GATED, MAP>>(a, units, stream);
    return launch_units<quant_kernel<__nv_bfloat16, GATED, MAP>>(a, units, stream);
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT int moe_quant_mxfp4(const void *x, int dtype, int64_t groups, int64_t rows, int64_t D,
                               uint8_t *codes, uint8_t *scales, moe_stream_t stream)
{
    MOE_TRACE("moe_quant_mxfp4");
    if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_EINVAL;
    if (check_tensor(groups, rows, D) != MOE_OK) return MOE_EINVAL;
    if (groups == 0 || rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_EINVAL;
    if (D % 32 || !aligned16(x) || !aligned16(codes) || !aligned4(scales)) return MOE_EALIGN;
    QuantArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.S = a.rows = groups * rows;
    a.D = D;
    a.group = rows;
    a.codes = codes;
    a.scales = reinterpret_cast<uint32_t *>(scales);
    return run_quant<false, false>(a, dtype, (cudaStream_t)stream);
}

MOE_EXPORT int moe_dispatch_quant_mxfp4(const void *x, int dtype, int64_t S, int64_t D, int K,
                                        const int64_t *tok_map, uint8_t *codes, uint8_t *scales,
                                        int64_t packed_rows, moe_stream_t stream)
{
    MOE_TRACE("moe_dispatch_quant_mxfp4");
    if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_EINVAL;
    if (S < 0 || K < 1 || K > 32 || S >= ((int64_t)1 << 31) / K) return MOE_EINVAL;
    if (check_tensor(1, packed_rows, D) != MOE_OK) return MOE_EINVAL;
    if (S == 0) return MOE_OK;
    if (packed_rows < 1 || !x || !tok_map || !codes || !scales) return MOE_EINVAL;
    if (D % 32 || !aligned16(x) || !aligned16(codes) || !aligned4(scales)) return MOE_EALIGN;
    QuantArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.map = tok_map;
    a.S = S;
    a.D = D;
    a.rows = a.group = packed_rows;
    a.K = K;
    a.codes = codes;
    a.scales = reinterpret_cast<uint32_t *>(scales);
    return run_quant<false, true>(a, dtype, (cudaStream_t)stream);
}

MOE_EXPORT int moe_swiglu_quant_mxfp4(const void *u, int dtype, int64_t rows, int64_t F,
                                      uint8_t *codes, uint8_t *scales, moe_stream_t stream)
{
    MOE_TRACE("moe_swiglu_quant_mxfp4");
    if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_EINVAL;
    if (check_tensor(1, rows, F) != MOE_OK) return MOE_EINVAL;
    if (rows == 0) return MOE_OK;
    if (!u || !codes || !scales) return MOE_EINVAL;
    if (F % 32 || !aligned16(u) || !aligned16(codes) || !aligned4(scales)) return MOE_EALIGN;
    QuantArgs a = {};
    a.x = static_cast<const uint8_t *>(u);
    a.S = a.rows = a.group = rows;
    a.D = F;
    a.codes = codes;
    a.scales = reinterpret_cast<uint32_t *>(scales);
    return run_quant<true, false>(a, dtype, (cudaStream_t)stream);
}

MOE_EXPORT int moe_dequant_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t groups,
                                 int64_t rows, int64_t D, void *out, int out_dtype,
                                 moe_stream_t stream)
{
    MOE_TRACE("moe_dequant_mxfp4");
    if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_EINVAL;
    if (check_tensor(groups, rows, D) != MOE_OK) return MOE_EINVAL;
    if (groups == 0 || rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return MOE_EINVAL;
    if (D % 32 || !aligned16(codes) || !aligned4(scales) || !aligned16(out)) return MOE_EALIGN;
    DequantArgs a = {codes, reinterpret_cast<const uint32_t *>(scales), groups * rows, D, rows,
                     static_cast<uint8_t *>(out)};
    return out_dtype == MOE_F32
               ? launch_units<dequant_kernel<float>>(a, units_of(a.rows, D, Dequant<float>::kUnit),
                                                     (cudaStream_t)stream)
               : launch_units<dequant_kernel<__nv_bfloat16>>(
                     a, units_of(a.rows, D, Dequant<__nv_bfloat16>::kUnit), (cudaStream_t)stream);
}

namespace moe {
// Reads and clears this file's device error bits.
cudaError_t read_mxfp4_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_mxfp4_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_mxfp4_error, &zero, sizeof(uint32_t));
    return e;
}
} // namespace moe
