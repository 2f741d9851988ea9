// A whole routed layer for a few tokens, weights in bf16 or MXFP4.
//
//   out[s] = sum_k topk_w[s,k] * w_down[e] h,   e = topk_idx[s,k]
//   h      = silu(w_gate[e] x[s]) * (w_up[e] x[s])
// with w_up [E, 2 F, H] (gates before ups) and w_down [E, H, F].  Every sum is f32; out
// is rounded once.
//
// Two launches (up, down), and one before them that prepares x for MXFP4 weights;
// each begins while the one before ends.  Up and down are one kernel.  Its CTAs, two
// an SM, walk tiles of 128 weight rows (64 gates and their ups; 128 outputs) for up
// to 8 entries (s, k) of an expert.  The weights bound the call: one token of 8
// experts reads 604 MB of bf16 weights or 160 MB of MXFP4, its other data are 100 KB.
// So one warp does nothing but copy weights with TMA into a ring of stages (80 or
// 64 KB of weights in flight a CTA), and begins before the launch waits for the one before
// it (nothing there writes weights).  A second warp copies the rows that they meet, one
// thread issues the matrix instructions (tcgen05, weights on the M side, entries on the N
// side: nothing is spent on a weight outside the tensor core), four warps read a tile's
// sums and four others the next one's.
// A token's outputs are summed over k by the CTA that brings the last of its experts.
// Tiles are dealt out in turn: taken from a counter, 32 tokens of 64 experts (7168, 2048,
// MXFP4) took 257 instead of 262 us, one token of 8 40 instead of 39.
//
// What it takes: one token of 8 experts (6144, 2048) 95 us in bf16 (6.3 TB/s of weights)
// and 38 us in MXFP4 (24 us of weights, and a chain of three launches: x is split after 4
// us, h is there after 29), 32 tokens of 64 experts (7168, 2048) in MXFP4 242 us (6.1
// TB/s).  With one group of storing warps 248 us, with one CTA an SM 12 % more.
//
// bf16 weights: x goes in as it is, a row an entry.  h is f32: it goes in as three
// bf16 rows that add up to it.
//
// MXFP4 weights: the block-scaled instruction (kind::mxf4) takes codes and scales as they
// are, but wants E2M1 on the other side too.  So x and h are written as sums of eight
// MXFP4 rows: of a block of 32 with largest magnitude a, 2^e <= a < 2^(e + 1), the first
// row is the block rounded to multiples of 2^(e - 1) and less (values up to 4 units,
// steps of at most one), the next what that left (at most half a unit) in units of
// 2^(e - 4), and so on, each three bits further.  The eighth leaves at most 2^-23 of a,
// about what an f32 sum does, or 2^-129 where the scales end.  Each row is a column of the
// product, and the columns' sums are added in f32.  Decoding the weights to f16 in registers
// for the warp-wide instruction instead takes 2.7 instructions a weight: 70 us for one token
// of 8 experts (6144, 2048) and 2290 us for 32 tokens of 64 (7168, 2048).
//
// The instruction wants the scales of 128 rows and 128 elements as words in 32 lanes
// x 4 columns of tensor memory, row 32 j + q in column j of lane q, and a copy from
// shared memory puts 16 bytes into one lane.  The rows' scales are written in that
// order here.  The weights' scales lie one word after another, so that their row
// 4 q + j arrives in column j of lane q, and TMA lays row 4 q + j of the codes in row 32 j
// + q of the stage to match (as in csrc/expert_gemm_mxfp4.cu).

#include "pair.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kMaxEntries = 1024;    // S * K
constexpr int kMaxExperts = 1024;
constexpr int kMaxWidth = 16384;     // H, F
constexpr int kThreads = 384;        // two groups of four storing warps take tiles by turns
constexpr int kSplitThreads = 256;
constexpr int kRows = 8;             // entries of a tile
constexpr int kTile = 128;           // weight rows of a tile
constexpr int kCodesA = kTile * 128; // of weights in a stage: 128 bytes of each row
constexpr int kScales = 2 * 512;     // of 128 rows in a stage, or places for them
constexpr int kMaxStages = 10;
constexpr int kScaleAt = 128;        // first TMEM column of the scales, after the accumulators
constexpr int kTmemCols = 256;       // so that two CTAs fit an SM
constexpr int kBoxBytes = 2 * kRows * kTile / 2 * 4;  // h of a tile of each group
// What depends on the weights' type: elements of a stage, rows that stand for one of h
// and the columns they take (one of x takes as many with MXFP4, one with bf16), bytes of
// the rows in a stage, and accumulators.
template <bool MX> struct Form;
template <> struct Form<true> {
    static constexpr int kK = 256, kH = 8, kColumns = 8, kAccs = 2;
    static constexpr int kCodesB = kRows * kColumns * 128;
    static constexpr int kStageBytes = kCodesA + kCodesB + 2 * kScales;
};
template <> struct Form<false> {
    static constexpr int kK = 64, kH = 3, kColumns = 4, kAccs = 4;
    static constexpr int kCodesB = kRows * kColumns * 128;
    static constexpr int kStageBytes = kCodesA + kCodesB;
};
constexpr int kParts = Form<true>::kH;

__device__ uint32_t g_layer_error;  // kErrExpertTimeout

// --- which experts have tokens ----------------------------------------------------

// Every CTA makes these lists for itself, in shared memory, from topk_idx: at most
// 1024 entries, 1 to 3 us, where a launch that makes them for all would cost as
// much.  Ranks are those of the entries' order, so all CTAs and launches agree.
struct Routing {
    int16_t *count;   // [E] an expert's place among those with tokens
    int16_t *hit;     // [hits] experts with tokens
    int16_t *first;   // [hits + 1] first packed row of each
    int16_t *parts;   // [hits + 1] parts of at most `rows` rows before each
    int16_t *order;   // [rows] the entry of each packed row
    int16_t *place;   // [S K] the row of each entry where parts have `rows` rows each, full
                      // or not; -1 without an expert
    int hits;

    static __host__ __device__ size_t bytes(int n, int E)
    {
        return (size_t)(E + 3 * (n < E ? n : E) + 2 + 2 * n) * 2;
    }

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

// `table`: THREADS / 32 x E counts in shared memory, for more than 32 entries.
template <int THREADS>
__device__ void route(const int32_t *idx, int n, int E, int rows, Routing &r, uint16_t *table)
{
    constexpr int kWarps = THREADS / 32, kEach = (kMaxExperts + THREADS - 1) / THREADS;
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
    // Each warp ranks neighbouring chunks of 32 entries; then the warps' counts of an
    // expert are added up in order.  (One warp alone takes 0.25 us a chunk.)
    const int each = ((n + 31) / 32 + kWarps - 1) / kWarps;  // chunks of a warp
    for (int i = tid; i < kWarps * E; i += THREADS) table[i] = 0;
    for (int i = tid; i < n; i += THREADS) {
        const int e = __ldg(idx + i);
        r.place[i] = e >= 0 && e < E ? e : -1;
    }
    __syncthreads();
    uint16_t *mine = table + warp * E;
    for (int i0 = warp * each * 32; i0 < min(n, (warp + 1) * each * 32); i0 += 32) {
        const int i = i0 + lane, e = i < n ? r.place[i] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int before = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0) {
            r.place[i] = before + __popc(same & lanemask_lt());
            if ((same & lanemask_lt()) == 0) mine[e] = before + __popc(same);
        }
        __syncwarp();
    }
    __syncthreads();
    // a thread owns kEach neighbouring experts
    int c[kEach], sum = 0, some = 0, part = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = tid * kEach + j;
        c[j] = 0;
        if (e < E)
            for (int w = 0; w < kWarps; ++w) {
                const int v = table[w * E + e];
                table[w * E + e] = (uint16_t)c[j];
                c[j] += v;
            }
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
            const int h = r.count[e], slot = table[i / (each * 32) * E + e] + r.place[i];
            r.order[r.first[h] + slot] = i;
            r.place[i] = r.parts[h] * rows + slot;
        }
    }
    fence_proxy_async_smem();  // the table's place may be copied into from here on
    __syncthreads();
}

// out[s, o .. o + 3] = sum over the valid entries of s, in increasing k, by a whole warp,
// each lane with its o: y [S K, H] holds the experts' rows by entry.  The loads are
// unconditional, so that eight are under way; a lane past the row reads its end.
__device__ __forceinline__ void sum_entries(const float *y, const float *topk_w,
                                            const int16_t *place, int K, int H, int o, int s,
                                            void *out, bool f32)
{
    constexpr int kAtOnce = 8;
    const int lane = threadIdx.x & 31, from = min(o, H - 4);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool mine = lane < K && place[s * K + lane] >= 0;  // K <= 32
    const float weight = mine ? __ldg(topk_w + s * K + lane) : 0.0f;
    const uint32_t valid = __ballot_sync(0xffffffffu, mine);
    for (int k0 = 0; k0 < K; k0 += kAtOnce) {
        float4 v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            v[k] = __ldcg(reinterpret_cast<const float4 *>(
                y + (int64_t)(s * K + min(k0 + k, K - 1)) * H + from));
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float w = __shfl_sync(0xffffffffu, weight, (k0 + k) & 31);
            // rows of entries without an expert hold anything
            if (k0 + k < K && (valid >> (k0 + k) & 1)) {
                sum.x = fmaf(w, v[k].x, sum.x);
                sum.y = fmaf(w, v[k].y, sum.y);
                sum.z = fmaf(w, v[k].z, sum.z);
                sum.w = fmaf(w, v[k].w, sum.w);
            }
        }
    }
    if (o >= H) return;
    const int64_t at = (int64_t)s * H + o;
    if (f32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = sum;
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y),
                             hi = __floats2bfloat162_rn(sum.z, sum.w);
        st8(static_cast<__nv_bfloat16 *>(out) + at,
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                       *reinterpret_cast<const uint32_t *>(&hi)));
    }
}

// --- x and h as eight rows ------------------------------------------------------

// Eight neighbouring values, four lanes a block of 32: the codes of row p (one
// word) and the block's scale byte.  `byte` is that of row 0, 255 where the block
// has an infinity or a NaN.  Rows whose scale would be below 2^-127 take that: what is
// left then is two units at most, of which the first of them leaves a quarter.
struct Split {
    float v[8];
    int byte;

    __device__ __forceinline__ void begin()
    {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = (int)(top >> 23);
        byte = e == 255 ? 255 : e - 1;  // -1 for zeros and what is below 2^-126
    }
    __device__ __forceinline__ int scale(int p) const
    {
        return byte == 255 ? (p ? 0 : 255) : max(byte - 3 * p, 0);  // E8M0 ends at 2^-127
    }
    __device__ __forceinline__ uint32_t next(int p)
    {
        if (byte == 255) return p ? 0 : 0x22222222u;  // ones, times NaN
        const uint32_t exponent = (uint32_t)max(byte - 3 * p, 0);
        const float inv = __uint_as_float((254u - exponent) << 23);
        const float unit = __uint_as_float(exponent ? exponent << 23 : 0x00400000u);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t code, back;
            asm("{\n\t.reg .b8 c;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 c, %3, %2;\n\t"
                "cvt.rn.f16x2.e2m1x2 %1, c;\n\t"
                "mov.b32 %0, {c, 0, 0, 0};\n\t}"
                : "=r"(code), "=r"(back)
                : "f"(v[2 * i] * inv), "f"(v[2 * i + 1] * inv));
            word |= (code & 255u) << (8 * i);
            const __half2 h = *reinterpret_cast<const __half2 *>(&back);
            // exact: what is left is a multiple of the value's last bit
            v[2 * i] = fmaf(-unit, __low2float(h), v[2 * i]);
            v[2 * i + 1] = fmaf(-unit, __high2float(h), v[2 * i + 1]);
        }
        return word;
    }
};

// Where the word of row p of an entry lies among the words of all parts.
__device__ __forceinline__ int scale_place(int place, int p)
{
    const int part = place / kRows, slot = place % kRows;  // column 8 slot + p = 32 j + q
    return part * 128 + (slot % 4 * kParts + p) * 4 + slot / 4;
}

struct SplitArgs {
    const uint8_t *x;
    const int32_t *idx;
    uint8_t *codes;      // [parts, 64, H / 2]
    uint32_t *scales;    // [ceil(H / 128), parts, 32, 4]
    int S, K, E, H, parts;
};

// A warp takes 256 elements of a token and stores them for its K entries.
__global__ void __launch_bounds__(kSplitThreads) split_kernel(SplitArgs a)
{
    extern __shared__ int16_t lists[];
    const int n = a.S * a.K;
    Routing rt(lists, n, a.E);
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    griddep_launch_dependents();
    route<kSplitThreads>(a.idx, n, a.E, kRows, rt,
                    reinterpret_cast<uint16_t *>(lists + Routing::bytes(n, a.E) / 2));
    const int chunks = (a.H + 255) / 256, words = (a.H + 127) / 128;
    for (int u = blockIdx.x * (kSplitThreads / 32) + (tid >> 5); u < a.S * chunks;
         u += gridDim.x * (kSplitThreads / 32)) {
        const int s = u / chunks, c = u - s * chunks, at = c * 256 + lane * 8;
        const bool in = at < a.H;
        Split sp;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = __ldg(reinterpret_cast<const uint4 *>(a.x + ((int64_t)s * a.H + at) * 2));
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sp.v[2 * k] = __uint_as_float(q[k] << 16);
            sp.v[2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
        }
        sp.begin();
        uint32_t code[kParts], word[kParts];
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            code[p] = sp.next(p);
            uint32_t b = (uint32_t)sp.scale(p);  // of four blocks, in every 16th lane
            b |= __shfl_down_sync(0xffffffffu, b, 4) << 8;
            word[p] = (b & 0xffffu) | __shfl_down_sync(0xffffffffu, b, 8) << 16;
        }
        const int w = 2 * c + (lane >> 4);
        uint32_t *scales = a.scales + (int64_t)w * a.parts * 128;
        for (int k = 0; k < a.K; ++k) {
            const int place = rt.place[s * a.K + k];
            if (place < 0) continue;
            uint8_t *codes = a.codes + (int64_t)place * kParts * (a.H / 2) + at / 2;
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                if (in) *reinterpret_cast<uint32_t *>(codes + p * (a.H / 2)) = code[p];
                if ((lane & 15) == 0 && w < words) scales[scale_place(place, p)] = word[p];
            }
        }
    }
}

// --- the products -----------------------------------------------------------------

struct LayerArgs {
    const int32_t *idx;
    const float *topk_w;
    uint8_t *h;           // MXFP4: codes [parts, 64, F / 2]; bf16 [parts, 32, F]
    uint8_t *h_scales;    // MXFP4: [ceil(F / 128), parts, 32, 4, 4]
    float *y;             // [n, H]
    uint32_t *arrived;    // [ceil(H / 128), S] experts whose share of these outputs is there
    uint8_t *out;
    int S, K, E, H, F;
    int parts;            // that there is room for
    int counters;
    int stages;
    int sum_stages;       // that are summed in tensor memory, the rest in registers
    int f32;
};

// The weights and the rows (of 4 entries, or 8; one of x for bf16), with MXFP4's
// scales.
struct LayerMaps {
    CUtensorMap a, sa, b[2], sb;
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void copy_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                        int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void copy_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                        int y)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
                 : "memory");
}

// Four rows of a map of single rows.
__device__ __forceinline__ void gather_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            const int (&row)[4])
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
                 ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]),
                 "r"(row[3])
                 : "memory");
}

__device__ __forceinline__ void copy_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                        int y, int z, int w)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void copy_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                        int y, int z, int w, int v)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
                 : "memory");
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t scale_a, uint32_t scale_b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void copy_scales(uint32_t d, uint64_t src)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(src) : "memory");
}

__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// Shared-memory descriptors: rows of 128 bytes under the 128-byte swizzle, and
// scales in rows of 16 bytes.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, bool rows)
{
    return ((uint64_t)(addr & 0x3ffff) >> 4) | (1ull << 16) |
           ((uint64_t)((rows ? 1024 : 128) >> 4) << 32) | (1ull << 46) |
           ((rows ? 2ull : 0ull) << 61);
}

// E2M1 operands, E8M0 scales; `half`: which two of a word's four scales.
__device__ __forceinline__ uint32_t instr_mxf4(int n, int half)
{
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           (1u << 23) | ((uint32_t)(kTile >> 4) << 24) | ((uint32_t)(2 * half) << 29);
}

// bf16 operands, f32 accumulator.
__device__ __forceinline__ uint32_t instr_bf16(int n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTile >> 4) << 24);
}

struct Tile {
    int e;        // expert
    int m;        // tile of its weights
    int part;     // of its entries
    int row;      // first packed row
    int rows;     // of them, 1 .. 8
};

// Tiles are numbered by part, then by the weights' tile, so that parts of one expert
// read the same weights one after another; asked for in order.
struct Walk {
    const Routing &rt;
    int tiles_m, at = 0;
    __device__ Walk(const Routing &r, int m) : rt(r), tiles_m(m) {}
    __device__ __forceinline__ Tile operator()(int t)
    {
        while (t >= rt.parts[at + 1] * tiles_m) ++at;
        const int parts = rt.parts[at + 1] - rt.parts[at];
        const int local = t - rt.parts[at] * tiles_m;
        Tile r;
        r.e = rt.hit[at];
        r.m = local / parts;
        r.part = rt.parts[at] + local - r.m * parts;
        r.row = rt.first[at] + (local - r.m * parts) * kRows;
        r.rows = min(kRows, rt.first[at + 1] - r.row);
        return r;
    }
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[4], acc_empty[4], drain;
    uint64_t turn[2];   // a group has read all accumulators of a tile
    uint32_t tmem;
    volatile int stop;
};

// A call, as its code in line costs calls without such gates up to 2 % (one or two tokens).
__device__ __noinline__ float rare_gate(float gate, float up) { return far_gate(gate, up); }

// h of a tile, 64 outputs of up to 8 entries in `box`, as the rows of the next product.
template <bool MX>
__device__ __forceinline__ void store_h(const LayerArgs &a, const Tile &c, const float *box, int me)
{
    if constexpr (MX) {
        // 4 threads a block, two blocks an entry
        const int x = me >> 3 & 7, b = me >> 2 & 1, l = me & 3;
        const int f0 = c.m * 64 + b * 32;
        if (me >= 64) return;
        Split sp;
#pragma unroll
        for (int k = 0; k < 8; ++k) sp.v[k] = x < c.rows ? box[x * 64 + b * 32 + l * 8 + k] : 0.0f;
        sp.begin();
        if (x >= c.rows || f0 >= a.F) return;
        const int place = c.part * kRows + x;
        uint8_t *codes = a.h + (int64_t)place * kParts * (a.F / 2) + f0 / 2 + l * 4;
        uint8_t *scales = a.h_scales + (int64_t)(f0 / 128) * a.parts * 512 + f0 / 32 % 4;
#pragma unroll 1
        for (int p = 0; p < kParts; ++p) {
            *reinterpret_cast<uint32_t *>(codes + p * (a.F / 2)) = sp.next(p);
            if (l == (p & 3)) {
                uint8_t *to = scales + scale_place(place, p) * 4;
                to[0] = (uint8_t)sp.scale(p);
                // the end of the last word
                if (f0 + 32 == a.F)
                    for (int k = 1; k <= 3 - f0 / 32 % 4; ++k) to[k] = 0;
            }
        }
    } else {
        // 16 threads an entry, four outputs each
        const int x = me >> 4, f = c.m * 64 + (me & 15) * 4;
        if (x >= c.rows || f >= a.F) return;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = box[x * 64 + (me & 15) * 4 + k];
        const int64_t row = (int64_t)(c.part * kRows + x) * Form<false>::kColumns;
#pragma unroll
        for (int p = 0; p < Form<false>::kH; ++p) {
            uint32_t u[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // cut, not rounded: three parts of 8 bits are the whole of an f32, and the
                // largest of them stay finite
                const __nv_bfloat162 b = __halves2bfloat162(__float2bfloat16_rz(v[2 * k]),
                                                            __float2bfloat16_rz(v[2 * k + 1]));
                u[k] = *reinterpret_cast<const uint32_t *>(&b);
                const float lo = __low2float(b), hi = __high2float(b);
                // nothing is left of an infinity
                v[2 * k] = isinf(lo) ? 0.0f : v[2 * k] - lo;
                v[2 * k + 1] = isinf(hi) ? 0.0f : v[2 * k + 1] - hi;
            }
            st8(a.h + ((row + p) * a.F + f) * 2, make_uint2(u[0], u[1]));
        }
    }
}

template <bool MX, bool UP>
__global__ void __launch_bounds__(kThreads, 2)
layer_kernel(const __grid_constant__ LayerMaps maps, LayerArgs a)
{
    using Fo = Form<MX>;
    constexpr int kAccs = Fo::kAccs, kAcc = kRows * Fo::kColumns;  // columns of one
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const int stages = a.stages;
    float *box = reinterpret_cast<float *>(ring + stages * Fo::kStageBytes);  // two of [8][64]
    const int n = a.S * a.K;
    int16_t *valid = reinterpret_cast<int16_t *>(box + kBoxBytes / 4);  // [S] experts of a token
    Routing rt(valid + a.S, n, a.E);
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 96) {
        prefetch_map(&maps.a);
        prefetch_map(&maps.b[0]);
        if (MX || !UP) prefetch_map(&maps.b[1]);
        if (MX) {
            prefetch_map(&maps.sa);
            prefetch_map(&maps.sb);
        }
    }
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh.full[i], 2);   // both operands
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 4);
        }
        mbar_init(&sh.turn[0], 4);
        mbar_init(&sh.turn[1], 4);
        mbar_init(&sh.drain, 1);
        sh.stop = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    // The first launch waits for what came before the call.  The others do so later:
    // topk_idx, topk_w and the experts' weights were complete when the first one began.
    constexpr bool kFirst = UP && !MX;
    if (kFirst) griddep_wait();
    route<kThreads>(a.idx, n, a.E, kRows, rt, reinterpret_cast<uint16_t *>(ring));  // has barriers
    if (!UP) {
        for (int s = tid; s < a.S; s += kThreads) {
            int k = 0;
            for (int i = s * a.K; i < (s + 1) * a.K; ++i) k += rt.place[i] >= 0;
            valid[s] = (int16_t)k;
        }
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int reduction = UP ? a.H : a.F, outputs = UP ? a.F : a.H;
    const int per_tile = UP ? kTile / 2 : kTile;
    const int tiles_m = (outputs + per_tile - 1) / per_tile;
    const int tiles = rt.parts[rt.hits] * tiles_m;
    const int blocks = (reduction + Fo::kK - 1) / Fo::kK;
    // columns of a tile of so many entries: those of 4 or 8; rows of x as they are take 8,
    // and 16 is the least there is
    auto columns_of = [&](int rows) {
        if (!MX && UP) return 16;
        return rows > kRows / 2 ? kRows * Fo::kColumns : kRows / 2 * Fo::kColumns;
    };
    Walk walk(rt, tiles_m);

    if (warp == 0 || warp == 2) {
        const bool is_weights = warp == 0;
        if (!is_weights && !kFirst) griddep_wait();  // the rows
        if (elect_one()) {
            Ring r(stages);
            int64_t j = 0;  // blocks copied
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile c = walk(t);
                const int cols = columns_of(c.rows);
                int token[2][4];  // rows of x, the last one again in the places of none
                if (!MX && UP && !is_weights)
#pragma unroll
                    for (int x = 0; x < kRows; ++x)
                        token[x / 4][x % 4] = rt.order[c.row + min(x, c.rows - 1)] / a.K;
                for (int b = 0; b < blocks; ++b, ++j) {
                    // the time until the launch before is done counts for no wait's limit
                    if (is_weights && !kFirst && j == stages) griddep_wait();
                    if (j >= stages && !wait(&sh.empty[r.at], r.round ^ 1, &sh.stop)) {
                        ok = false;
                        break;
                    }
                    uint8_t *stage = ring + r.at * Fo::kStageBytes;
                    uint8_t *rows = stage + kCodesA, *scales = rows + Fo::kCodesB;
                    uint64_t *bar = &sh.full[r.at];
                    const int m = c.m * per_tile;
                    if (is_weights) {
                        mbar_arrive_expect_tx(bar, kCodesA + (MX ? kScales : 0));
                        if (MX && UP) {
                            // 64 gates and 64 ups: row 4 q + j of either in lane
                            // 32 j + q, ups 16 lanes on
                            copy_5d(stage, &maps.a, bar, b * 128, m / 4, 0, 0, c.e);
                            copy_4d(scales, &maps.sa, bar, m, 0, 2 * b, c.e);
                        } else if (MX) {
                            copy_4d(stage, &maps.a, bar, b * 128, m / 4, 0, c.e);
                            copy_3d(scales, &maps.sa, bar, m, 2 * b, c.e);
                        } else if (UP) {
                            // gates 8 i .. in lanes 16 i .., their ups 8 lanes on
                            copy_5d(stage, &maps.a, bar, b * 64, 0, 0, m / 8, c.e);
                        } else {
                            copy_3d(stage, &maps.a, bar, b * 64, m, c.e);
                        }
                    } else if (!MX && UP) {
                        // Four rows a copy: with one each, 16 tokens of 2 of 8 experts
                        // (5120, 832) took 76 us instead of 55.
                        mbar_arrive_expect_tx(bar, c.rows == 1 ? 128 : c.rows > 4 ? 1024 : 512);
                        if (c.rows == 1) copy_2d(rows, &maps.b[0], bar, b * 64, token[0][0]);
                        else gather_rows(rows, &maps.b[0], bar, b * 64, token[0]);
                        if (c.rows > 4) gather_rows(rows + 512, &maps.b[0], bar, b * 64, token[1]);
                    } else {
                        mbar_arrive_expect_tx(bar, cols * 128 + (MX ? kScales : 0));
                        copy_2d(rows, &maps.b[c.rows > kRows / 2], bar, b * (MX ? 128 : 64),
                                c.part * (kRows * Fo::kColumns));
                        if (MX) copy_2d(scales + kScales, &maps.sb, bar, c.part * 128, 2 * b);
                    }
                    r.next();
                }
            }
            if (!ok) {
                // leave no copy in flight
                for (int64_t i = j > stages ? j - stages : 0; i < j; ++i)
                    (void)wait_slow(&sh.full[i % stages], (uint32_t)(i / stages) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // One thread issues.  A stage has its own columns of scales: the copy into it,
        // which begins when the products that read it before are done, frees both.
        if (!kFirst) griddep_wait();
        if (elect_one()) {
            Ring r(stages);
            int i = 0;  // accumulators begun
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int cols = columns_of(walk(t).rows);
                const uint32_t low = MX ? instr_mxf4(cols, 0) : instr_bf16(cols);
                const uint32_t high = instr_mxf4(cols, 1);
                uint32_t acc = 0;
                int next = 0;  // first block of the next accumulator
                for (int b = 0; b < blocks; ++b) {
                    const bool fresh = b == next;  // a division here costs 3 % of a call
                    if (fresh) {
                        next += a.sum_stages;
                        if (b > 0) commit(&sh.acc_full[(i - 1) % kAccs]);
                        const int at = i % kAccs;
                        if (i >= kAccs &&
                            !wait(&sh.acc_empty[at], (uint32_t)(i / kAccs - 1) & 1, &sh.stop)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        acc = tmem + at * kAcc;
                        ++i;
                    }
                    if (!wait(&sh.full[r.at], r.round, &sh.stop)) {
                        ok = false;
                        break;
                    }
                    const uint32_t stage = smem_u32(ring) + r.at * Fo::kStageBytes;
                    tc_fence_after();
                    const uint64_t da = desc_of(stage, true), db = da + (kCodesA >> 4);
                    const int left = reduction - b * Fo::kK;  // a quarter of a stage a product
                    if constexpr (MX) {
                        const uint32_t sa = tmem + kScaleAt + (uint32_t)r.at * 16, sb = sa + 8;
                        const uint64_t from_a = desc_of(stage + kCodesA + Fo::kCodesB, false);
                        const uint64_t from_b = from_a + (kScales >> 4);
                        copy_scales(sa, from_a);
                        copy_scales(sb, from_b);
                        mma_mxf4(acc, da, db, low, sa, sb, !fresh);
                        if (left > 64) mma_mxf4(acc, da + 2, db + 2, high, sa, sb, true);
                        if (left > 128) {
                            copy_scales(sa + 4, from_a + 32);
                            copy_scales(sb + 4, from_b + 32);
                            mma_mxf4(acc, da + 4, db + 4, low, sa + 4, sb + 4, true);
                            if (left > 192)
                                mma_mxf4(acc, da + 6, db + 6, high, sa + 4, sb + 4, true);
                        }
                    } else {
                        mma_bf16(acc, da, db, low, !fresh);
                        if (left > 16) mma_bf16(acc, da + 2, db + 2, low, true);
                        if (left > 32) mma_bf16(acc, da + 4, db + 4, low, true);
                        if (left > 48) mma_bf16(acc, da + 6, db + 6, low, true);
                    }
                    commit(&sh.empty[r.at]);
                    r.next();
                }
                if (ok) commit(&sh.acc_full[(i - 1) % kAccs]);
            }
            commit(&sh.drain);  // nothing is issued after this
        }
        __syncwarp();
    } else if (warp >= 4) {
        // this warp's quarter and group; of the group's 128 threads
        const int q = warp & 3, group = (warp - 4) >> 2, me = (tid - 128) & 127;
        box += group * (kBoxBytes / 8);
        auto join = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
        // whether all four warps go on: one that gave up must not leave the others
        // at their next meeting; the meeting is one of whole warps
        auto agree = [&](bool ok) {
            uint32_t all;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\t"
                         "setp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, %2, 128, p;\n\t"
                         "selp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"((uint32_t)ok), "r"(1 + group)
                         : "memory");
            return all != 0;
        };
        if (!kFirst) griddep_wait();
        griddep_launch_dependents();
        if (UP) {
            for (int i = blockIdx.x * 256 + tid - 128; i < a.counters; i += gridDim.x * 256)
                a.arrived[i] = 0;
        } else {
            // tokens without an expert
            for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
                if (valid[s]) continue;
                for (int i = tid - 128; i < a.H; i += 256) {
                    if (a.f32) reinterpret_cast<float *>(a.out)[(int64_t)s * a.H + i] = 0.0f;
                    else reinterpret_cast<uint16_t *>(a.out)[(int64_t)s * a.H + i] = 0;
                }
            }
        }
        const int accumulators = (blocks + a.sum_stages - 1) / a.sum_stages;  // of a tile
        int i = group * accumulators, taken = 0;
        for (int t = blockIdx.x + group * gridDim.x; t < tiles;
             t += 2 * gridDim.x, i += accumulators, ++taken) {
            const Tile c = walk(t);
            float sum[kRows];
#pragma unroll
            for (int x = 0; x < kRows; ++x) sum[x] = 0.0f;
            // Not before the other group has read the tile before: a barrier that is
            // rounds behind would look as if this round were done.
            const int turns = taken - 1 + group;
            bool ok = turns < 0 || wait_warp(&sh.turn[group ^ 1], (uint32_t)turns & 1, &sh.stop);
            for (int b = 0; b < blocks && ok; b += a.sum_stages, ++i) {
                const int buf = i % kAccs;
                ok = wait_warp(&sh.acc_full[buf], (uint32_t)(i / kAccs) & 1, &sh.stop);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kAcc;
                if constexpr (MX) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j * 4 >= c.rows) break;
                        uint32_t v[32];  // column 8 x + p: row p of entry 4 j + x
                        tmem_load(acc + j * 32, v);
                        tmem_wait(v);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float f = __uint_as_float(v[8 * x + 7]);  // the small ones first
#pragma unroll
                            for (int p = 6; p >= 0; --p) f += __uint_as_float(v[8 * x + p]);
                            sum[4 * j + x] += f;
                        }
                    }
                } else if constexpr (UP) {
                    uint32_t v[16];
                    tmem_load(acc, v);
                    tmem_wait(v);
#pragma unroll
                    for (int x = 0; x < kRows; ++x) sum[x] += __uint_as_float(v[x]);
                } else {
                    uint32_t v[32];  // column 4 x + p
                    tmem_load(acc, v);
                    tmem_wait(v);
#pragma unroll
                    for (int x = 0; x < kRows; ++x)
                        sum[x] += (__uint_as_float(v[4 * x + 2]) + __uint_as_float(v[4 * x + 1])) +
                                  __uint_as_float(v[4 * x]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            }
            if (lane == 0) mbar_arrive(&sh.turn[group]);
            if (!agree(ok)) break;
            if constexpr (UP) {
                // the gate of an output here, its up 16 (or 8) lanes on
                const bool gate = MX ? lane < 16 : (lane & 8) == 0;
                const int f = MX ? 4 * lane + q : 16 * q + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                for (int x = 0; x < kRows; ++x) {
                    const float up = __shfl_down_sync(0xffffffffu, sum[x], MX ? 16 : 8);
                    if (gate && x < c.rows)
                        box[x * 64 + f] = sum[x] < kFarGate
                                              ? rare_gate(sum[x], up)
                                              : sum[x] / (1.0f + expf(-sum[x])) * up;
                }
                join();
                store_h<MX>(a, c, box, me);
                join();  // the box has been read
            } else {
                // A token's outputs are summed by the CTA that brings the last of its
                // experts, which spreads the sums over the call (by the last expert's CTA
                // for all tokens they took 55 us at the end of 32), by a warp all 128 of
                // them: little code, which a call's end meets for the first time.
                const int o = c.m * kTile + (MX ? 4 * lane + q : 32 * q + lane);
                if (o < a.H)
#pragma unroll
                    for (int x = 0; x < kRows; ++x)
                        if (x < c.rows) a.y[(int64_t)rt.order[c.row + x] * a.H + o] = sum[x];
                join();
                __threadfence();  // of all four warps' stores, which the join has ordered
                int token = 0;
                bool last = false;
                if (lane < 2 && q + 4 * lane < c.rows) {  // entries q and q + 4
                    token = rt.order[c.row + q + 4 * lane] / a.K;
                    last = atomicAdd(a.arrived + c.m * a.S + token, 1u) + 1 ==
                           (uint32_t)valid[token];
                }
                uint32_t ready = __ballot_sync(0xffffffffu, last);
                if (ready) {
                    __threadfence();
                    __syncwarp();  // what the counting lanes saw, all lanes may read
                }
                for (; ready; ready &= ready - 1) {
                    const int s = __shfl_sync(0xffffffffu, token, __ffs(ready) - 1);
                    sum_entries(a.y, a.topk_w, rt.place, a.K, a.H, c.m * kTile + 4 * lane, s,
                                a.out, a.f32);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        (void)wait_slow(&sh.drain, 0, nullptr);  // the last matrix instruction
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols));
    }
    if (tid == 0 && sh.stop) atomicOr(&g_layer_error, kErrExpertTimeout);
}

// --- host ----------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

struct Shape {
    int rank;
    cuuint64_t dims[5], strides[4];   // strides of all but the innermost, in bytes
    cuuint32_t box[5];
};

cudaError_t encode(CUtensorMap *map, const void *base, CUtensorMapDataType type, const Shape &s)
{
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    const bool words = type == CU_TENSOR_MAP_DATA_TYPE_UINT32;  // scales
    const CUresult r =
        fn(map, type, s.rank, const_cast<void *>(base), s.dims, s.strides, s.box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           words ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr CUtensorMapDataType kBytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapDataType kWords = CU_TENSOR_MAP_DATA_TYPE_UINT32;
constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// Shared memory of one of two CTAs in an SM, which has 228 KB and keeps 1 KB for each,
// less what the kernel declares: its barriers, and three sums of each warp from the ranking.
constexpr size_t kSmem =
    (228 << 10) / 2 - 1024 - sizeof(Shared) - 3 * (kThreads / 32) * sizeof(int);

struct LaunchShape {
    int stages, ctas;   // ctas: of an SM
    size_t smem;
    int64_t tiles;      // at most
};

template <bool MX, bool UP> LaunchShape launch_shape(const LayerArgs &a)
{
    constexpr int kStageBytes = Form<MX>::kStageBytes;
    const size_t rest = 1024 + kBoxBytes + a.S * 2 + Routing::bytes(a.S * a.K, a.E);
    const int per_tile = UP ? kTile / 2 : kTile;
    LaunchShape r;
    r.tiles = (int64_t)(((UP ? a.F : a.H) + per_tile - 1) / per_tile) * a.parts;
    // Two CTAs of an SM have four or five stages each.  Where the lists leave less, or
    // there is no work for two, one CTA has more of them (5 tokens of 24 experts, 1416,
    // 520, bf16: 21.1 -> 19.1 us).
    const int least = MX ? 4 : 5;
    r.stages = (int)((kSmem - rest) / kStageBytes);
    r.ctas = r.stages < least || r.tiles <= sm_count() ? 1 : 2;
    if (r.ctas == 1) r.stages = MX ? 7 : 9;
    r.smem = rest + (size_t)r.stages * kStageBytes;
    return r;
}

template <bool MX, bool UP>
int launch_layer(const LayerMaps &maps, LayerArgs a, cudaStream_t stream)
{
    static KernelCache kc;
    const LaunchShape l = launch_shape<MX, UP>(a);
    a.stages = l.stages;
    cudaError_t e = prepare_kernel(layer_kernel<MX, UP>, l.smem, kThreads, kc, nullptr);
    if (e == cudaSuccess) {
        const int64_t room = (int64_t)sm_count() * l.ctas;
        e = launch_pdl(layer_kernel<MX, UP>, dim3((unsigned)(l.tiles < room ? l.tiles : room)),
                       dim3(kThreads), l.smem, stream, maps, a);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

// The CTAs of an SM that a call's launch counts on, and those that fit one by their shared
// memory, registers, threads and tensor memory.  (The runtime's own count of CTAs is 1 for
// any kernel that allocates tensor memory.)
template <bool MX, bool UP> int launch_ctas(const LayerArgs &a, int32_t *counts)
{
    const LaunchShape l = launch_shape<MX, UP>(a);
    cudaFuncAttributes f;
    int dev = 0, smem = 0, kept = 0, regs = 0, threads = 0;
    cudaError_t e = cudaFuncGetAttributes(&f, layer_kernel<MX, UP>);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    auto ask = [&](int *v, cudaDeviceAttr attr) {
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(v, attr, dev);
    };
    ask(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor);
    ask(&kept, cudaDevAttrReservedSharedMemoryPerBlock);
    ask(&regs, cudaDevAttrMaxRegistersPerMultiprocessor);
    ask(&threads, cudaDevAttrMaxThreadsPerMultiProcessor);
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    int64_t most = smem / (round_up(f.sharedSizeBytes + l.smem, 128) + kept);
    const int64_t limits[3] = {regs / (round_up(f.numRegs, 8) * kThreads), threads / kThreads,
                               512 / kTmemCols};
    for (int64_t v : limits) most = v < most ? v : most;
    counts[0] = l.ctas;
    counts[1] = (int32_t)most;
    return MOE_OK;
}

// Parts of n entries: one for every eight of an expert and one for what is left.
int64_t most_parts(int64_t n, int64_t E) { return n < E + n / kRows ? n : E + n / kRows; }

// The workspace: x and h as rows of the products, y, and the counters.
struct Places {
    int64_t x, x_scales, h, h_scales, y, arrived, bytes;
    Places(bool mx, int64_t S, int64_t K, int64_t E, int64_t H, int64_t F)
    {
        const int64_t n = S * K, parts = most_parts(n, E);
        int64_t at = 0;
        auto take = [&](int64_t size) {
            const int64_t p = at;
            at += round_up(size, 256);
            return p;
        };
        x = take(mx ? parts * kRows * kParts * H / 2 : 0);
        x_scales = take(mx ? (H + 127) / 128 * parts * 512 : 0);
        h = take(parts * kRows * (mx ? kParts * F / 2 : Form<false>::kColumns * F * 2));
        h_scales = take(mx ? (F + 127) / 128 * parts * 512 : 0);
        y = take(n * H * 4);
        arrived = take(counters(S, H) * 4);
        bytes = at;
    }
    static int64_t counters(int64_t S, int64_t H) { return (H + kTile - 1) / kTile * S; }
};

struct LayerCall {
    const uint8_t *x, *up, *up_scales, *down, *down_scales;
    uint8_t *workspace;
};

// Parts of 64 rows of D elements as the other operand of MXFP4 weights.
cudaError_t encode_mx_rows(LayerMaps &m, const uint8_t *codes, const uint8_t *scales, int parts,
                           int D)
{
    const cuuint64_t row = D / 2, P = parts, words = (D + 127) / 128;
    constexpr cuuint32_t kCols = kRows * kParts;
    cudaError_t e = cudaSuccess;
    for (cuuint32_t i = 0; i < 2 && e == cudaSuccess; ++i)
        e = encode(&m.b[i], codes, kBytes, {2, {row, P * kCols}, {row}, {128, kCols / 2 * (i + 1)}});
    if (e != cudaSuccess) return e;
    return encode(&m.sb, scales, kWords, {2, {P * 128, words}, {P * 512}, {128, 2}});
}

int layer_mxfp4(const LayerCall &c, LayerArgs a, cudaStream_t stream)
{
    const Places at(true, a.S, a.K, a.E, a.H, a.F);
    uint8_t *ws = c.workspace;
    a.h = ws + at.h;
    a.h_scales = ws + at.h_scales;
    // Products of E2M1 are whole numbers under their scales, and sums of them lose nothing
    // while all terms lie within 24 bits of the largest sum.  Where a row's scales are spread
    // further, each step of 64 cuts the sum's low bits off: over 16384 elements with scales of
    // 2^20 that left 9e-6 of the result (2-norm), with sums of 16 steps in f32 outputs 7e-7,
    // as plain f32 sums have; it costs 0 to 1 % (8 experts of 4096, 1024 with 64 tokens each:
    // 60 -> 61.5 us).
    a.sum_stages = a.f32 ? 4 : kMaxWidth / Form<true>::kK;
    a.y = reinterpret_cast<float *>(ws + at.y);
    a.arrived = reinterpret_cast<uint32_t *>(ws + at.arrived);
    LayerMaps up = {}, down = {};
    const cuuint64_t E = a.E, H = a.H, F = a.F;
    const cuuint64_t up_row = H / 2, up_words = (H + 127) / 128;
    const cuuint64_t down_row = F / 2, down_words = (F + 127) / 128;
    // gates and ups as two runs of F rows
    cudaError_t e = encode(&up.a, c.up, kBytes,
                           {5,
                            {up_row, F / 4, 2, 4, E},
                            {4 * up_row, F * up_row, up_row, 2 * F * up_row},
                            {128, 16, 2, 4, 1}});
    if (e == cudaSuccess)
        e = encode(&up.sa, c.up_scales, kWords,
                   {4, {F, 2, up_words, E}, {F * 4, 2 * F * 4, up_words * 2 * F * 4}, {64, 2, 2, 1}});
    if (e == cudaSuccess) e = encode_mx_rows(up, ws + at.x, ws + at.x_scales, a.parts, a.H);
    if (e == cudaSuccess)
        e = encode(&down.a, c.down, kBytes,
                   {4, {down_row, H / 4, 4, E}, {4 * down_row, down_row, H * down_row}, {128, 32, 4, 1}});
    if (e == cudaSuccess)
        e = encode(&down.sa, c.down_scales, kWords,
                   {3, {H, down_words, E}, {H * 4, down_words * H * 4}, {kTile, 2, 1}});
    if (e == cudaSuccess) e = encode_mx_rows(down, a.h, a.h_scales, a.parts, a.F);
    static KernelCache kc;
    const size_t smem = Routing::bytes(a.S * a.K, a.E) + (size_t)a.E * (kSplitThreads / 32) * 2;
    if (e == cudaSuccess) e = prepare_kernel(split_kernel, smem, kSplitThreads, kc, nullptr);
    if (e == cudaSuccess) {
        const SplitArgs s = {c.x, a.idx, ws + at.x, reinterpret_cast<uint32_t *>(ws + at.x_scales),
                             a.S, a.K, a.E, a.H, a.parts};
        const int64_t units = (int64_t)a.S * ((a.H + 255) / 256), most = 2 * sm_count();
        const int64_t grid = (units + kSplitThreads / 32 - 1) / (kSplitThreads / 32);
        e = launch_pdl(split_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(kSplitThreads),
                       smem, stream, s);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    int r = check_launch();
    if (r == MOE_OK) r = launch_layer<true, true>(up, a, stream);
    if (r == MOE_OK) r = launch_layer<true, false>(down, a, stream);
    return r;
}

int layer_bf16(const LayerCall &c, LayerArgs a, cudaStream_t stream)
{
    const Places at(false, a.S, a.K, a.E, a.H, a.F);
    a.h = c.workspace + at.h;
    a.y = reinterpret_cast<float *>(c.workspace + at.y);
    a.arrived = reinterpret_cast<uint32_t *>(c.workspace + at.arrived);
    LayerMaps up = {}, down = {};
    const cuuint64_t E = a.E, H = a.H, F = a.F, P = a.parts;
    constexpr cuuint32_t kCols = kRows * Form<false>::kColumns;
    // gates and ups as two runs of F rows, eight of either by turns
    cudaError_t e = encode(&up.a, c.up, kBf16,
                           {5,
                            {H, 8, 2, F / 8, E},
                            {H * 2, F * H * 2, 8 * H * 2, 2 * F * H * 2},
                            {64, 8, 2, 8, 1}});
    if (e == cudaSuccess)
        e = encode(&up.b[0], c.x, kBf16, {2, {H, (cuuint64_t)a.S}, {H * 2}, {64, 1}});
    if (e == cudaSuccess)
        e = encode(&down.a, c.down, kBf16, {3, {F, H, E}, {F * 2, H * F * 2}, {64, kTile, 1}});
    for (cuuint32_t i = 0; i < 2 && e == cudaSuccess; ++i)
        e = encode(&down.b[i], a.h, kBf16, {2, {F, P * kCols}, {F * 2}, {64, kCols / 2 * (i + 1)}});
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    // The tensor core cuts a sum's low bits off at each step of 16: f32 outputs are off
    // by 2e-6 after 48 of them and 4e-7 after 8, for 4 % of time (one token of 8 experts,
    // 6144, 2048: 95 and 99 us).
    a.sum_stages = a.f32 ? 2 : 12;
    const int r = launch_layer<false, true>(up, a, stream);
    return r == MOE_OK ? launch_layer<false, false>(down, a, stream) : r;
}

bool in_range(int64_t S, int64_t H, int K, int E, int64_t F)
{
    return S >= 0 && K >= 1 && K <= 32 && E >= 1 && E <= kMaxExperts && H >= 1 && F >= 1 &&
           H <= kMaxWidth && F <= kMaxWidth && S <= kMaxEntries && S * K <= kMaxEntries;
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT size_t moe_expert_layer_workspace_size(int64_t S, int64_t H, int K, int E, int64_t F,
                                                  int w_dtype)
{
    if (!in_range(S, H, K, E, F) || (w_dtype != MOE_BF16 && w_dtype != MOE_MXFP4)) return 0;
    return (size_t)Places(w_dtype == MOE_MXFP4, S, K, E, H, F).bytes;
}

MOE_EXPORT int moe_selftest_layer_ctas(int64_t S, int64_t H, int K, int E, int64_t F, int w_dtype,
                                       int32_t *counts)
{
    if (!in_range(S, H, K, E, F) || S < 1 || (w_dtype != MOE_BF16 && w_dtype != MOE_MXFP4) || !counts)
        return MOE_EINVAL;
    LayerArgs a = {};
    a.S = (int)S;
    a.K = K;
    a.E = E;
    a.H = (int)H;
    a.F = (int)F;
    a.parts = (int)most_parts(S * K, E);
    const bool mx = w_dtype == MOE_MXFP4;
    const int r = mx ? launch_ctas<true, true>(a, counts) : launch_ctas<false, true>(a, counts);
    if (r != MOE_OK) return r;
    return mx ? launch_ctas<true, false>(a, counts + 2) : launch_ctas<false, false>(a, counts + 2);
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
    if (workspace_bytes < moe_expert_layer_workspace_size(S, H, K, E, F, w_dtype))
        return MOE_EINVAL;
    const int step = mx ? 32 : 8;
    if (H % step || F % step || !aligned16(x) || !aligned16(w_up) || !aligned16(w_down) ||
        !aligned16(out) || !aligned16(workspace) ||
        (mx && (!aligned16(up_scales) || !aligned16(down_scales))))
        return MOE_EALIGN;
    LayerArgs a = {};
    a.idx = topk_idx;
    a.topk_w = topk_w;
    a.out = static_cast<uint8_t *>(out);
    a.S = (int)S;
    a.K = K;
    a.E = E;
    a.H = (int)H;
    a.F = (int)F;
    a.parts = (int)most_parts(S * K, E);
    a.counters = (int)Places::counters(S, H);
    a.f32 = f32;
    const LayerCall c = {static_cast<const uint8_t *>(x),
                         static_cast<const uint8_t *>(w_up),
                         up_scales,
                         static_cast<const uint8_t *>(w_down),
                         down_scales,
                         static_cast<uint8_t *>(workspace)};
    return mx ? layer_mxfp4(c, a, (cudaStream_t)stream) : layer_bf16(c, a, (cudaStream_t)stream);
}

namespace moe {
// Reads and clears this file's device error bits.
cudaError_t read_layer_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_layer_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_layer_error, &zero, sizeof(uint32_t));
    return e;
}
} // namespace moe
