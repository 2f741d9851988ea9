// A whole routed layer for a few tokens, in two launches.
//
//   out[s] = sum_k topk_w[s,k] * w_down[e] h,   e = topk_idx[s,k]
//   h      = silu(w_gate[e] x[s]) * (w_up[e] x[s])
// with w_up [E, 2 F, H] (gates before ups) and w_down [E, H, F] in bf16 or MXFP4
// (csrc/mxfp4.cu has the format).  Every sum is f32; out is rounded once.
//
// The first launch writes h of every entry (s, k), the second y = w_down h, and
// the CTA that brings the last expert's share of 32 columns sums them over k.
// Both list the experts that have tokens from topk_idx (every CTA for itself), cut
// their weights into tiles of 32 rows and hand each CTA a contiguous run of them.
//
// A tile's weights are read once, straight into registers, and bound the call: one
// token of 8 experts reads 604 MB of bf16 weights, its other data are 100 KB.  The
// eight warps of a CTA share the reduction, each 1/8 of it over all 32 rows, and
// add their sums in shared memory, in order.  A lane's next loads are issued before it
// uses the last ones, across tiles, so that the reads do not stop while the warps
// meet.  The products are those of the warp-wide matrix instruction (mma.sync,
// 16 x 8 x 16): with at most a few tokens an expert it is far from bounding, and it
// takes weights from registers, where MXFP4 is decoded.
//
// bf16: lane (g, t) holds 8 elements of rows g and g + 8 and the eight columns are
// tokens.  x goes in as it is.  h has more bits than bf16: it goes in as two bf16 parts
// (16 bits; three parts for f32 outputs), each a column, whose sums are added.
//
// MXFP4: lane (g, t) holds block t of 128 elements of rows g and g + 8, so the four
// blocks, which have a scale each, lie in the four lanes that an instruction sums
// over.  The columns keep them apart: column 2 b + j holds token j's elements of
// block b and zeros in the lanes of the others, which makes column 2 t + j, in lane t, the sum of
// block t for token j.  It is scaled there, by the one scale that this lane has read.
// Codes are decoded to f16 (exactly); x and h go in as f16 times a power of two
// that brings the largest of a row's slice to 2^14 .. 2^15: bf16 values keep all
// bits down to 2^-28 of the largest and 2^-39 of it after that; h keeps 11 bits, or
// 22 in two parts for f32 outputs.

#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;            // weight rows of a tile: two of the instruction's 16
constexpr int kDepth = 2;            // chunks of 64 bytes of each row in flight
constexpr int kMaxRows = 8;          // tokens of an expert taken at once
constexpr int kMaxEntries = 1024;    // S * K
constexpr int kMaxExperts = 1024;
constexpr int kMaxWidth = 16384;     // H, F
constexpr int kStageBudget = 88 << 10;  // so that two CTAs fit an SM

struct LayerArgs {
    const uint8_t *x;        // bf16 [S, H]
    const int32_t *idx;      // [S, K]
    const float *topk_w;     // [S, K]
    const uint8_t *w;        // this launch's weights (codes)
    const uint8_t *scales;   // MXFP4
    float *h;                // [S K, F]
    float *y;                // [S K, H]
    uint32_t *arrived;       // [ceil(H / 32)] experts whose share of these columns is there
    uint8_t *out;            // [S, H]
    int S, K, E, H, F;
    int rows;                // tokens of an expert taken at once
    int pitch;               // bytes of a staged row of one warp
    int out_f32;
};

// What a row of x or h becomes in shared memory, and how many such rows the
// instruction's eight columns hold.
template <bool MX, int PARTS> struct Staged {
    static constexpr int kChunk = MX ? 128 : 32;           // elements of 64 bytes of weights
    static constexpr int kChunkBytes = kChunk * 2;
    static constexpr int kRows = MX ? 2 / PARTS : 8 / (PARTS == 3 ? 4 : PARTS);
    static constexpr int kStride = PARTS == 3 ? 4 : PARTS; // columns (slots) of a row
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1, bool half)
{
    if (half)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight codes of a word as four pairs of f16.
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&f)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
        : "r"(w));
}

// 2^(byte - 127); NaN for 255
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return __uint_as_float(byte == 255 ? 0x7fffffffu : byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The experts that have tokens and whose they are.
struct Routing {
    int *count;   // [E], then the first entry of each expert in `order`
    int *hit;     // [hits] experts with tokens, in increasing order
    int *order;   // [S K] entries by expert
    int hits;
};

__device__ void route(const LayerArgs &a, Routing &r)
{
    __shared__ int s_sum[kWarps], s_hits[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.S * a.K;
    constexpr int kEach = kMaxEntries / kThreads, kExperts = kMaxExperts / kThreads;
    for (int e = tid; e < a.E; e += kThreads) r.count[e] = 0;
    __syncthreads();
    int e_of[kEach], slot[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = tid + j * kThreads;
        e_of[j] = i < n ? __ldg(a.idx + i) : -1;
        if (e_of[j] < 0 || e_of[j] >= a.E) e_of[j] = -1;
        // any order will do: tokens of an expert do not meet in a sum
        if (e_of[j] >= 0) slot[j] = atomicAdd(&r.count[e_of[j]], 1);
    }
    __syncthreads();
    // thread tid owns experts tid * kExperts ..
    int c[kExperts], sum = 0, some = 0;
#pragma unroll
    for (int j = 0; j < kExperts; ++j) {
        const int e = tid * kExperts + j;
        c[j] = e < a.E ? r.count[e] : 0;
        sum += c[j];
        some += c[j] > 0;
    }
    int upto = sum, hits = some;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o), v = __shfl_up_sync(0xffffffffu, hits, o);
        if (lane >= o) {
            upto += u;
            hits += v;
        }
    }
    if (lane == 31) {
        s_sum[warp] = upto;
        s_hits[warp] = hits;
    }
    __syncthreads();
    int first = upto - sum, at = hits - some;
    r.hits = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            first += s_sum[w];
            at += s_hits[w];
        }
        r.hits += s_hits[w];
    }
#pragma unroll
    for (int j = 0; j < kExperts; ++j) {
        const int e = tid * kExperts + j;
        if (e < a.E) r.count[e] = first;
        if (c[j] > 0) r.hit[at++] = e;
        first += c[j];
    }
    if (tid == kThreads - 1) r.count[a.E] = first;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (e_of[j] >= 0) r.order[r.count[e_of[j]] + slot[j]] = tid + j * kThreads;
    __syncthreads();
}

// Eight neighbouring values of a row of x or h as f32; zeros past the row.
template <bool UP>
__device__ __forceinline__ void load8(const LayerArgs &a, int entry, int k, int K, float (&f)[8])
{
    if (k >= K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    } else if (UP) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(
            a.x + ((int64_t)(entry / a.K) * K + k) * 2));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(a.h + (int64_t)entry * K + k);
        const float4 u = __ldcg(p), v = __ldcg(p + 1);
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
        f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
    }
}

// One warp's slice (elements from .. from + len of K) of up to `rows` entries.
template <bool MX, bool UP, int PARTS>
__device__ void stage(const LayerArgs &a, const int *entries, int rows, int from, int len, int K,
                      uint8_t *to, float *back)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int r = 0; r < rows; ++r) {
        const int entry = entries[r];
        float up = 1.0f, up2 = 1.0f;
        if (MX) {
            // 2^(14 - e) in two factors, e the exponent of the largest finite value
            uint32_t top = 0;
            for (int k = lane * 8; k < len; k += 256) {
                float f[8];
                load8<UP>(a, entry, from + k, K, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t m = __float_as_uint(f[i]) & 0x7fffffffu;
                    if (m < 0x7f800000u) top = max(top, m);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = 141 - (int)(top >> 23);  // 14 - (exponent), -113 .. 141
            const int half = e >> 1;
            up = __uint_as_float((uint32_t)(127 + half) << 23);
            up2 = __uint_as_float((uint32_t)(127 + e - half) << 23);
            // 2^-e: subnormal below 2^-126
            if (lane == 0)
                back[r] = e > 126 ? __uint_as_float(1u << (149 - e))
                                  : __uint_as_float((uint32_t)(127 - e) << 23);
        }
        uint8_t *p = to + r * PARTS * a.pitch;
        for (int k = lane * 8; k < len; k += 256) {
            float f[8];
            load8<UP>(a, entry, from + k, K, f);
            if (MX)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * up * up2;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = MX ? pack_half(f[2 * i], f[2 * i + 1]) : pack_bf16(f[2 * i], f[2 * i + 1]);
                    if (part + 1 < PARTS) {
                        float lo, hi;
                        if (MX) {
                            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                            lo = v.x, hi = v.y;
                        } else {
                            lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xffff0000u);
                        }
                        // nothing is left of an infinity
                        f[2 * i] = isinf(lo) ? 0.0f : f[2 * i] - lo;
                        f[2 * i + 1] = isinf(hi) ? 0.0f : f[2 * i + 1] - hi;
                    }
                }
                *reinterpret_cast<uint4 *>(p + part * a.pitch + k * 2) =
                    make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
    __syncwarp();
}

// A place in the CTA's run of tiles: the next 64 bytes of each of a tile's rows.
struct Cursor {
    int item, pass, chunk;
};

template <bool MX, bool UP, int PARTS, int NT>
__global__ void __launch_bounds__(kThreads, 2) layer_kernel(LayerArgs a)
{
    using St = Staged<MX, PARTS>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n = a.S * a.K;
    // shared memory: staged rows, the warps' sums (twice), scales back, the routing
    const int staged_rows = a.rows * PARTS;
    uint8_t *mine = smem + warp * staged_rows * a.pitch;
    float *sums = reinterpret_cast<float *>(smem + kWarps * staged_rows * a.pitch);
    float *back = sums + 2 * kWarps * kMaxRows * kTile;
    int *lists = reinterpret_cast<int *>(back + kWarps * kMaxRows);
    Routing rt = {lists, lists + a.E + 1, lists + a.E + 1 + min(n, a.E), 0};
    __shared__ int s_last;

    const int K = UP ? a.H : a.F;                    // reduction
    const int M = UP ? 2 * a.F : a.H;                // weight rows of an expert
    const int per_tile = UP ? kTile / 2 : kTile;     // outputs of a tile
    const int outputs = UP ? a.F : a.H;
    const int tiles = (outputs + per_tile - 1) / per_tile;
    const int row_bytes = MX ? K / 2 : K * 2;
    const int chunks = (row_bytes + 63) / 64;
    const int c0 = chunks * warp / kWarps, mc = chunks * (warp + 1) / kWarps - c0;
    const int steps = max(mc, 1);                    // a warp without chunks takes part

    if (UP) {
        griddep_wait();
        griddep_launch_dependents();
        const int columns = (a.H + kTile - 1) / kTile;
        for (int i = blockIdx.x * kThreads + tid; i < columns; i += gridDim.x * kThreads)
            a.arrived[i] = 0;
    }
    // The second launch lists and begins to read its weights while the first one
    // ends: what it reads until its wait was complete when that one began.
    route(a, rt);
    const int64_t items = (int64_t)rt.hits * tiles;
    const int begin = (int)(items * blockIdx.x / gridDim.x);
    const int end = (int)(items * (blockIdx.x + 1) / gridDim.x);

    auto tokens_of = [&](int item) {
        const int e = rt.hit[item / tiles];
        return rt.count[e + 1] - rt.count[e];
    };
    auto passes_of = [&](int item) { return (tokens_of(item) + a.rows - 1) / a.rows; };
    auto advance = [&](Cursor &c, int len) {
        if (++c.chunk < len) return false;
        c.chunk = 0;
        if (++c.pass == passes_of(c.item)) {
            c.pass = 0;
            ++c.item;
        }
        return true;
    };

    // --- loads ---
    uint4 w[kDepth][4];     // rows g, g + 8 of both halves of the tile
    uint32_t sc[kDepth];    // their scales' bytes
    Cursor ahead = {begin, 0, 0};
    const uint8_t *from = nullptr, *scale_from = nullptr;
    uint32_t ok = 0;        // which of the four rows exist
    const int64_t half = (int64_t)(UP ? a.F : kTile / 2);  // rows between the halves
    auto aim = [&] {
        if (ahead.item >= end) return;
        const int h = ahead.item / tiles, e = rt.hit[h];
        const int row = (ahead.item - h * tiles) * per_tile + g;
        ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row + (i & 1) * 8 + (UP ? 0 : (i >> 1) * (kTile / 2));
            if (r < outputs) ok |= 1u << i;
        }
        from = a.w + ((int64_t)e * M + row) * row_bytes + c0 * 64 + t * 16;
        if (MX)
            scale_from = a.scales + (((int64_t)e * chunks + c0) * M + row) * 4 + t;
    };
    auto load = [&](int d) {
        const int at = (c0 + ahead.chunk) * 64 + t * 16;
        const bool in = ahead.item < end && ahead.chunk < mc && at < row_bytes;
        sc[d] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = (i & 1) * 8 + (i >> 1) * half;
            w[d][i] = make_uint4(0, 0, 0, 0);
            if (in && (ok >> i & 1)) {
                w[d][i] = ld_stream16(from + r * row_bytes + ahead.chunk * 64);
                if (MX)
                    sc[d] |= (uint32_t)__ldg(scale_from + (r + (int64_t)ahead.chunk * M) * 4) << (8 * i);
            }
        }
        if (ahead.item < end && advance(ahead, steps)) aim();
    };
    aim();
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(d);

    if (!UP) {
        griddep_wait();  // h and the cleared counters
        griddep_launch_dependents();
        if (rt.hits == 0) {
            for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < (int64_t)a.S * a.H;
                 i += (int64_t)gridDim.x * kThreads) {
                if (a.out_f32) reinterpret_cast<float *>(a.out)[i] = 0.0f;
                else reinterpret_cast<uint16_t *>(a.out)[i] = 0;
            }
            return;
        }
    }

    // --- products ---
    float acc[2][NT][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
    };
    clear();
    Cursor now = {begin, 0, 0};
    int staged_e = -1, staged_pass = 0;
    int e = 0, first = 0, rows = 0, need = 0;  // of this visit
    int turn = 0;
    auto visit = [&] {
        if (now.item >= end) return;
        e = rt.hit[now.item / tiles];
        first = rt.count[e] + now.pass * a.rows;
        rows = min(a.rows, rt.count[e + 1] - first);
        need = (rows + St::kRows - 1) / St::kRows;
        if (e != staged_e || now.pass != staged_pass) {
            stage<MX, UP, PARTS>(a, rt.order + first, rows, c0 * St::kChunk, mc * St::kChunk, K,
                                 mine, back + warp * kMaxRows);
            staged_e = e;
            staged_pass = now.pass;
        }
    };
    visit();

    auto products = [&](int d) {
        if (now.chunk >= mc) return;
        const uint8_t *b0 = mine + now.chunk * St::kChunkBytes;
        if constexpr (!MX) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= need) break;
                // column g: part g % kStride of row g / kStride, or a column that is not used
                const int row = j * St::kRows + g / St::kStride, part = g % St::kStride;
                uint4 b = make_uint4(0, 0, 0, 0);
                if (row < rows && part < PARTS)
                    b = *reinterpret_cast<const uint4 *>(b0 + (row * PARTS + part) * a.pitch + t * 16);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint4 u = w[d][2 * m], v = w[d][2 * m + 1];
                    mma(acc[m][j], u.x, v.x, u.y, v.y, b.x, b.y, false);
                    mma(acc[m][j], u.z, v.z, u.w, v.w, b.z, b.w, false);
                }
            }
        } else {
            constexpr int kAtOnce = NT < 2 ? NT : 2;
            float s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = scale_of(sc[d] >> (8 * i) & 255u);
            const bool holds = t == g >> 1;  // this lane's elements of block t, slot g & 1
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += kAtOnce) {
                if (j0 >= need) break;
                float c[2][kAtOnce][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[m][j][i] = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 b[kAtOnce];
#pragma unroll
                    for (int j = 0; j < kAtOnce; ++j) {
                        const int slot = (j0 + j) * 2 + (g & 1);
                        b[j] = make_uint4(0, 0, 0, 0);
                        if (holds && slot < rows * PARTS)
                            b[j] = *reinterpret_cast<const uint4 *>(b0 + slot * a.pitch + t * 64 + q * 16);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint4 lo = w[d][2 * m], hi = w[d][2 * m + 1];
                        uint32_t u[4], v[4];
                        decode(q == 0 ? lo.x : q == 1 ? lo.y : q == 2 ? lo.z : lo.w, u);
                        decode(q == 0 ? hi.x : q == 1 ? hi.y : q == 2 ? hi.z : hi.w, v);
#pragma unroll
                        for (int j = 0; j < kAtOnce; ++j) {
                            mma(c[m][j], u[0], v[0], u[1], v[1], b[j].x, b[j].y, true);
                            mma(c[m][j], u[2], v[2], u[3], v[3], b[j].z, b[j].w, true);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    // rows of the two slots; those past the last are not used
                    const float *p = back + warp * kMaxRows;
                    const float f0 = p[min(((j0 + j) * 2) / PARTS, rows - 1)];
                    const float f1 = p[min(((j0 + j) * 2 + 1) / PARTS, rows - 1)];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[m][j0 + j][i] =
                                fmaf(s[2 * m + (i >> 1)], c[m][j][i] * (i & 1 ? f1 : f0), acc[m][j0 + j][i]);
                }
            }
        }
    };

    // The warps' sums meet; a thread finishes one output.
    auto finish = [&] {
        float *to = sums + (turn * kWarps + warp) * kMaxRows * kTile;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j >= need) break;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = acc[m][j][i];
                    if (MX) {  // over the four blocks
                        v[i] += __shfl_xor_sync(0xffffffffu, v[i], 1);
                        v[i] += __shfl_xor_sync(0xffffffffu, v[i], 2);
                    }
                }
                const int at = m * 16 + g;
                if (MX) {
                    if (PARTS == 2) {
                        if (t == 0 && j < rows) {
                            to[j * kTile + at] = v[0] + v[1];
                            to[j * kTile + at + 8] = v[2] + v[3];
                        }
                    } else if (t < 2 && 2 * j + t < rows) {
                        to[(2 * j + t) * kTile + at] = t ? v[1] : v[0];
                        to[(2 * j + t) * kTile + at + 8] = t ? v[3] : v[2];
                    }
                } else if (PARTS == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = j * 8 + 2 * t + (i & 1);
                        if (row < rows) to[row * kTile + at + (i >> 1) * 8] = v[i];
                    }
                } else if (PARTS == 2) {
                    const int row = j * 4 + t;
                    if (row < rows) {
                        to[row * kTile + at] = v[0] + v[1];
                        to[row * kTile + at + 8] = v[2] + v[3];
                    }
                } else {  // columns 4 row .. 4 row + 2
                    const float u0 = v[0] + v[1], u1 = v[2] + v[3];
                    const float w0 = u0 + __shfl_xor_sync(0xffffffffu, u0, 1);
                    const float w1 = u1 + __shfl_xor_sync(0xffffffffu, u1, 1);
                    const int row = j * 2 + (t >> 1);
                    if ((t & 1) == 0 && row < rows) {
                        to[row * kTile + at] = w0;
                        to[row * kTile + at + 8] = w1;
                    }
                }
            }
        }
        clear();
        __syncthreads();
        const float *p = sums + turn * kWarps * kMaxRows * kTile;
        turn ^= 1;
        const int o0 = now.item % tiles * per_tile;
        const int at = tid % per_tile, row = tid / per_tile;
        if (row < rows && o0 + at < outputs) {
            const int entry = rt.order[first + row];
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                v[0] += p[(k * kMaxRows + row) * kTile + at];
                if (UP) v[1] += p[(k * kMaxRows + row) * kTile + kTile / 2 + at];
            }
            if (UP) a.h[(int64_t)entry * a.F + o0 + at] = v[0] / (1.0f + expf(-v[0])) * v[1];
            else a.y[(int64_t)entry * a.H + o0 + at] = v[0];
        }
    };

    // The last expert's CTA for 32 columns sums them over each token's entries.
    auto combine = [&](int item) {
        const int tile = item % tiles, o = tile * kTile + (tid & 31);
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(a.arrived + tile, 1u) == (uint32_t)rt.hits - 1;
            __threadfence();
        }
        __syncthreads();
        if (!s_last || o >= a.H) return;
        for (int s = warp; s < a.S; s += kWarps) {
            float sum = 0.0f;
            for (int k = 0; k < a.K; ++k) {
                const int i = s * a.K + k, id = __ldg(a.idx + i);
                if (id >= 0 && id < a.E)
                    sum += __ldg(a.topk_w + i) * __ldcg(a.y + (int64_t)i * a.H + o);
            }
            if (a.out_f32) reinterpret_cast<float *>(a.out)[(int64_t)s * a.H + o] = sum;
            else
                reinterpret_cast<__nv_bfloat16 *>(a.out)[(int64_t)s * a.H + o] =
                    __float2bfloat16_rn(sum);
        }
    };

    while (now.item < end) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (now.item >= end) break;
            products(d);
            load(d);
            if (now.chunk + 1 == steps) {
                finish();
                const int item = now.item;
                advance(now, steps);
                if (!UP && now.item != item) combine(item);
                visit();
            } else {
                ++now.chunk;
            }
        }
    }
}

// --- host ----------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

template <bool MX, bool UP, int PARTS, int NT>
int launch_layer(LayerArgs a, cudaStream_t stream)
{
    static KernelCache kc;
    using St = Staged<MX, PARTS>;
    auto kernel = layer_kernel<MX, UP, PARTS, NT>;
    const int K = UP ? a.H : a.F, n = a.S * a.K;
    const int chunks = ((MX ? K / 2 : K * 2) + 63) / 64;
    const int mine = (chunks + kWarps - 1) / kWarps;  // of one warp
    // neighbouring staged rows begin in other banks
    a.pitch = mine * St::kChunkBytes;
    a.pitch += ((MX ? 32 : 64) - a.pitch % 128 + 128) % 128;
    const int row = kWarps * PARTS * a.pitch;
    int rows = kStageBudget / row;
    const int most = NT * St::kRows < kMaxRows ? NT * St::kRows : kMaxRows;
    if (rows > most) rows = most;
    if (rows > a.S) rows = a.S;
    a.rows = rows < 1 ? 1 : rows;
    const size_t smem = (size_t)a.rows * row + 2 * kWarps * kMaxRows * kTile * 4 +
                        kWarps * kMaxRows * 4 + ((size_t)a.E + 1 + (n < a.E ? n : a.E) + n) * 4;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(kernel, smem, kThreads, kc, &per_sm);
    if (e == cudaSuccess) {
        const int per_tile = UP ? kTile / 2 : kTile;
        const int64_t tiles = ((UP ? a.F : a.H) + per_tile - 1) / per_tile;
        const int64_t items = tiles * (n < a.E ? n : a.E);
        const int64_t most_ctas = (int64_t)sm_count() * (per_sm < 1 ? 1 : per_sm);
        e = launch_pdl(kernel, dim3((unsigned)(items < most_ctas ? items : most_ctas)),
                       dim3(kThreads), smem, stream, a);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

bool in_range(int64_t S, int64_t H, int K, int E, int64_t F)
{
    return S >= 0 && K >= 1 && K <= 32 && E >= 1 && E <= kMaxExperts && H >= 1 && F >= 1 &&
           H <= kMaxWidth && F <= kMaxWidth && S <= kMaxEntries && S * K <= kMaxEntries;
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT size_t moe_expert_layer_workspace_size(int64_t S, int64_t H, int K, int E, int64_t F)
{
    if (!in_range(S, H, K, E, F)) return 0;
    return (size_t)(round_up(S * K * H * 4, 256) + round_up(S * K * F * 4, 256) +
                    round_up((H + kTile - 1) / kTile * 4, 256));
}

MOE_EXPORT int moe_expert_layer(const void *x, int64_t S, int64_t H, const int32_t *topk_idx,
                                const float *topk_w, int K, int E, int64_t F, int w_dtype,
                                const void *w_up, const uint8_t *up_scales, const void *w_down,
                                const uint8_t *down_scales, void *out, int out_dtype,
                                void *workspace, size_t workspace_bytes, moe_stream_t stream)
{
    MOE_TRACE("moe_expert_layer");
    const bool mx = w_dtype == MOE_MXFP4, f32 = out_dtype == MOE_F32;
    if ((w_dtype != MOE_BF16 && !mx) || (out_dtype != MOE_BF16 && !f32)) return MOE_EINVAL;
    if (!in_range(S, H, K, E, F)) return MOE_EINVAL;
    if (S == 0) return MOE_OK;
    if (!x || !topk_idx || !topk_w || !w_up || !w_down || !out || !workspace) return MOE_EINVAL;
    if (mx && (!up_scales || !down_scales)) return MOE_EINVAL;
    if (workspace_bytes < moe_expert_layer_workspace_size(S, H, K, E, F)) return MOE_EINVAL;
    const int step = mx ? 32 : 8;
    if (H % step || F % step || !aligned16(x) || !aligned16(w_up) || !aligned16(w_down) ||
        !aligned16(out) || !aligned16(workspace))
        return MOE_EALIGN;
    LayerArgs a = {};
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.x = static_cast<const uint8_t *>(x);
    a.idx = topk_idx;
    a.topk_w = topk_w;
    a.w = static_cast<const uint8_t *>(w_up);
    a.scales = up_scales;
    a.y = reinterpret_cast<float *>(ws);
    ws += round_up(S * K * H * 4, 256);
    a.h = reinterpret_cast<float *>(ws);
    ws += round_up(S * K * F * 4, 256);
    a.arrived = reinterpret_cast<uint32_t *>(ws);
    a.out = static_cast<uint8_t *>(out);
    a.S = (int)S;
    a.K = K;
    a.E = E;
    a.H = (int)H;
    a.F = (int)F;
    a.out_f32 = f32;
    const cudaStream_t st = (cudaStream_t)stream;
    LayerArgs b = a;
    b.w = static_cast<const uint8_t *>(w_down);
    b.scales = down_scales;
    int r;
    if (!mx) {
        r = launch_layer<false, true, 1, 1>(a, st);
        if (r != MOE_OK) return r;
        return f32 ? launch_layer<false, false, 3, 4>(b, st) : launch_layer<false, false, 2, 2>(b, st);
    }
    if (S <= 2) {
        r = launch_layer<true, true, 1, 1>(a, st);
        if (r != MOE_OK) return r;
        return f32 ? launch_layer<true, false, 2, 2>(b, st) : launch_layer<true, false, 1, 1>(b, st);
    }
    r = launch_layer<true, true, 1, 4>(a, st);
    if (r != MOE_OK) return r;
    return f32 ? launch_layer<true, false, 2, 4>(b, st) : launch_layer<true, false, 1, 4>(b, st);
}
