// A whole routed layer for a few tokens on MXFP4 weights.
//
//   out[s] = sum_k topk_w[s,k] * w_down[e] h,   e = topk_idx[s,k]
//   h      = silu(w_gate[e] x[s]) * (w_up[e] x[s])
//
// The weights bound the call, and the block-scaled matrix instruction
// (kind::mxf4) takes them as they are, with no instruction spent on a weight;
// decoding them in registers for mma.sync takes 2.7 instructions a weight and ran at
// 2.3 TB/s.  The other operand has to be E2M1 too, so x and h are written as sums of
// eight MXFP4 rows: of a block of 32 with largest magnitude a, 2^e <= a < 2^(e + 1),
// the first row is the block rounded to multiples of 2^(e - 1) and less (values up
// to 4 units, steps of at most one), the next what that left (at most half a unit) in units of 2^(e - 4),
// and so on, each three bits further.  The eighth leaves at most 2^-23 of a, less than f32 sums do.
// Each row is a column of the product, and the columns' sums are added in f32.
//
// Three launches, each of which begins while the one before ends:
//   split  x of every entry to eight rows, ordered by expert
//   up     gates and ups of 64 outputs for up to 8 entries of an expert (64 columns),
//          the activation, and h to eight rows
//   down   128 outputs for up to 8 entries; a token's are summed over k as the last of
//          its experts arrives
// Up and down are one kernel: CTAs, two an SM, walk tiles of 128 weight rows.  One
// warp copies weights with TMA, one the rows, into a ring of stages of 256 elements, a
// third issues the products, four more read the sums.  The copies of weights begin
// before the launch waits for the one before it: nothing there writes weights.
//
// The instruction wants the scales of 128 rows and 128 elements as words in 32 lanes
// x 4 columns of tensor memory, row 32 j + q in column j of lane q, and a copy from
// shared memory puts 16 bytes into one lane.  The rows' scales are written in that
// order here.  The weights' scales lie one word after another, so that their row
// 4 q + j arrives in column j of lane q, and TMA lays row 4 q + j of the codes in row 32 j
// + q of the stage to match (as in csrc/expert_gemm_mxfp4.cu).

#include "few.cuh"
#include "pair.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 8;            // rows that stand for one
constexpr int kRows = 8;             // entries of a tile
constexpr int kCols = kRows * kParts;
constexpr int kTile = 128;           // weight rows of a tile
constexpr int kK = 256;              // elements of a stage
constexpr int kCodesA = kTile * kK / 2;
constexpr int kCodesB = kCols * kK / 2;
constexpr int kScales = 2 * 512;     // of 128 rows, or places for them
constexpr int kStageBytes = kCodesA + kCodesB + 2 * kScales;
constexpr int kMaxStages = 7;
constexpr int kScaleAt = 2 * kCols;  // first TMEM column of the scales
constexpr int kTmemCols = 256;       // so that two CTAs fit an SM
constexpr int kSmem = 115712;        // of shared memory, likewise
constexpr int kBoxBytes = kRows * kTile / 2 * 4;  // h of a tile

__device__ uint32_t g_layer_error;  // kErrExpertTimeout

// --- x and h as eight rows ------------------------------------------------------

// Eight neighbouring values, four lanes a block of 32: the codes of row p (one
// word) and the block's scale byte.  `byte` is that of row 0, 255 where the block
// has an infinity or a NaN; rows whose scale would be below 2^-127 are zero.
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
        return byte == 255 ? (p ? 0 : 255) : max(byte - 3 * p, 0);
    }
    __device__ __forceinline__ uint32_t next(int p)
    {
        if (byte == 255) return p ? 0 : 0x22222222u;  // ones, times NaN
        if (byte - 3 * p < 0) return 0;
        const float inv = __uint_as_float((uint32_t)(254 - (byte - 3 * p)) << 23);
        const float unit = byte - 3 * p ? __uint_as_float((uint32_t)(byte - 3 * p) << 23)
                                        : __uint_as_float(0x00400000u);
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
    uint32_t *arrived;   // cleared for the third launch
    int S, K, E, H, parts, counters;
};

// A warp takes 256 elements of a token and stores them for its K entries.
__global__ void __launch_bounds__(kThreads) split_kernel(SplitArgs a)
{
    extern __shared__ int16_t lists[];
    const int n = a.S * a.K;
    Routing rt(lists, n, a.E);
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    griddep_launch_dependents();
    for (int i = blockIdx.x * kThreads + tid; i < a.counters; i += gridDim.x * kThreads)
        a.arrived[i] = 0;
    route<kThreads>(a.idx, n, a.E, kRows, rt);
    const int chunks = (a.H + 255) / 256, words = (a.H + 127) / 128;
    for (int u = blockIdx.x * (kThreads / 32) + (tid >> 5); u < a.S * chunks;
         u += gridDim.x * (kThreads / 32)) {
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
    uint8_t *h_codes;     // [parts, 64, F / 2]
    uint8_t *h_scales;    // [ceil(F / 128), parts, 32, 4, 4]
    float *y;             // [n, H]
    uint32_t *arrived;    // [ceil(H / 128), 4, S] experts whose share of these outputs is there
    uint8_t *out;
    int S, K, E, H, F;
    int parts;            // that there is room for
    int stages;
    int f32;
};

// Codes and scales of the weights and of the rows (of 4 entries, or 8).
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

// Shared-memory descriptors: codes in rows of 128 bytes under the 128-byte swizzle,
// scales in rows of 16 bytes.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, bool codes)
{
    return ((uint64_t)(addr & 0x3ffff) >> 4) | (1ull << 16) |
           ((uint64_t)((codes ? 1024 : 128) >> 4) << 32) | (1ull << 46) |
           ((codes ? 2ull : 0ull) << 61);
}

// E2M1 operands, E8M0 scales; `half`: which two of a word's four scales.
__device__ __forceinline__ uint32_t instr_desc(int n, int half)
{
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           (1u << 23) | ((uint32_t)(kTile >> 4) << 24) | ((uint32_t)(2 * half) << 29);
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
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    volatile int stop;
};

template <bool UP>
__global__ void __launch_bounds__(kThreads, 2)
layer_kernel(const __grid_constant__ LayerMaps maps, LayerArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const int stages = a.stages;
    float *box = reinterpret_cast<float *>(ring + stages * kStageBytes);  // [8][64]
    const int n = a.S * a.K;
    float *weights = box + kBoxBytes / 4;                       // [n]
    int16_t *valid = reinterpret_cast<int16_t *>(weights + n);  // [S] experts of a token
    Routing rt(valid + a.S, n, a.E);
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 96) {
        prefetch_map(&maps.a);
        prefetch_map(&maps.sa);
        prefetch_map(&maps.b[0]);
        prefetch_map(&maps.b[1]);
        prefetch_map(&maps.sb);
    }
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh.full[i], 2);   // both operands
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 4);
        }
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
    // topk_idx, topk_w and the experts' weights were complete when the first launch began
    if (!UP) load_weights(a.topk_w, n, weights);
    route<kThreads>(a.idx, n, a.E, kRows, rt);  // begins and ends with a barrier
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
    const int blocks = (reduction + kK - 1) / kK;
    Walk walk(rt, tiles_m);

    if (warp == 0 || warp == 2) {
        const bool weights = warp == 0;
        if (!weights) griddep_wait();  // the rows
        if (elect_one()) {
            Ring r(stages);
            int64_t j = 0;  // blocks copied
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile c = walk(t);
                const bool all = c.rows > kRows / 2;
                for (int b = 0; b < blocks; ++b, ++j) {
                    if (j >= stages && !wait(&sh.empty[r.at], r.round ^ 1, &sh.stop)) {
                        ok = false;
                        break;
                    }
                    uint8_t *stage = ring + r.at * kStageBytes;
                    uint64_t *bar = &sh.full[r.at];
                    if (weights) {
                        mbar_arrive_expect_tx(bar, kCodesA + kScales);
                        const int m = c.m * per_tile;
                        uint8_t *scales = stage + kCodesA + kCodesB;
                        if (UP) {
                            // 64 gates and 64 ups: row 4 q + j of either in lane
                            // 32 j + q, ups 16 lanes on
                            copy_5d(stage, &maps.a, bar, b * 128, m / 4, 0, 0, c.e);
                            copy_4d(scales, &maps.sa, bar, m, 0, 2 * b, c.e);
                        } else {
                            copy_4d(stage, &maps.a, bar, b * 128, m / 4, 0, c.e);
                            copy_3d(scales, &maps.sa, bar, m, 2 * b, c.e);
                        }
                    } else {
                        mbar_arrive_expect_tx(bar, kCodesB / (all ? 1 : 2) + kScales);
                        copy_2d(stage + kCodesA, &maps.b[all], bar, b * 128, c.part * kCols);
                        copy_2d(stage + kCodesA + kCodesB + kScales, &maps.sb, bar, c.part * 128,
                                2 * b);
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
        if (elect_one()) {
            Ring r(stages);
            int i = 0;  // tiles begun
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++i) {
                const int cols = walk(t).rows > kRows / 2 ? kCols : kCols / 2;
                const uint32_t low = instr_desc(cols, 0), high = instr_desc(cols, 1);
                if (i >= 2 && !wait(&sh.acc_empty[i & 1], (uint32_t)(i / 2 - 1) & 1, &sh.stop))
                    break;
                tc_fence_after();
                const uint32_t acc = tmem + (i & 1) * kCols;
                for (int b = 0; b < blocks; ++b) {
                    if (!wait(&sh.full[r.at], r.round, &sh.stop)) {
                        ok = false;
                        break;
                    }
                    const uint32_t stage = smem_u32(ring) + r.at * kStageBytes;
                    tc_fence_after();
                    const uint32_t sa = tmem + kScaleAt + (uint32_t)r.at * 16, sb = sa + 8;
                    const uint64_t from_a = desc_of(stage + kCodesA + kCodesB, false);
                    const uint64_t from_b = from_a + (kScales >> 4);
                    const uint64_t da = desc_of(stage, true), db = da + (kCodesA >> 4);
                    const int left = reduction - b * kK;  // 64 elements a product
                    copy_scales(sa, from_a);
                    copy_scales(sb, from_b);
                    mma_mxf4(acc, da, db, low, sa, sb, b > 0);
                    if (left > 64) mma_mxf4(acc, da + 2, db + 2, high, sa, sb, true);
                    if (left > 128) {
                        copy_scales(sa + 4, from_a + 32);
                        copy_scales(sb + 4, from_b + 32);
                        mma_mxf4(acc, da + 4, db + 4, low, sa + 4, sb + 4, true);
                        if (left > 192) mma_mxf4(acc, da + 6, db + 6, high, sa + 4, sb + 4, true);
                    }
                    commit(&sh.empty[r.at]);
                    r.next();
                }
                if (ok) commit(&sh.acc_full[i & 1]);
            }
            commit(&sh.drain);  // nothing is issued after this
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int q = warp & 3, me = tid - 128;  // this warp's quarter; of 128 threads
        auto join = [&] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        // whether all four warps go on: one that gave up must not leave the others
        // at their next meeting
        auto agree = [&](bool ok) {
            uint32_t all;
            asm volatile("{\n\t.reg .pred p, q;\n\t"
                         "setp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, 1, 128, p;\n\t"
                         "selp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"((uint32_t)ok)
                         : "memory");
            return all != 0;
        };
        griddep_wait();
        griddep_launch_dependents();
        if (!UP) {
            // tokens without an expert
            for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
                if (valid[s]) continue;
                for (int i = me; i < a.H; i += 128) {
                    if (a.f32) reinterpret_cast<float *>(a.out)[(int64_t)s * a.H + i] = 0.0f;
                    else reinterpret_cast<uint16_t *>(a.out)[(int64_t)s * a.H + i] = 0;
                }
            }
        }
        int i = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            const Tile c = walk(t);
            const int buf = i & 1;
            if (!agree(wait(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop))) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kCols;
            float sum[kRows];
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
                    sum[4 * j + x] = f;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            if constexpr (UP) {
                // lane q of a quarter j: gate of output 4 q + j, lane 16 + q its up
#pragma unroll
                for (int x = 0; x < kRows; ++x) {
                    const float up = __shfl_down_sync(0xffffffffu, sum[x], 16);
                    if (lane < 16 && x < c.rows)
                        box[x * 64 + 4 * lane + q] = sum[x] / (1.0f + expf(-sum[x])) * up;
                }
                join();
                // 4 threads a block, two blocks an entry
                const int x = me >> 3 & 7, b = me >> 2 & 1, l = me & 3;
                const int f0 = c.m * 64 + b * 32;
                if (me < 64) {
                    Split sp;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sp.v[k] = x < c.rows ? box[x * 64 + b * 32 + l * 8 + k] : 0.0f;
                    sp.begin();
                    if (x < c.rows && f0 < a.F) {
                        const int place = c.part * kRows + x;
                        uint8_t *codes = a.h_codes + (int64_t)place * kParts * (a.F / 2) +
                                         f0 / 2 + l * 4;
                        uint8_t *scales = a.h_scales + (int64_t)(f0 / 128) * a.parts * 512 +
                                          f0 / 32 % 4;
#pragma unroll
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
                    }
                }
                join();  // the box has been read
            } else {
                // Each warp stores its outputs (every fourth) and counts them for
                // itself: the warps need not meet.  A token's outputs are summed by the
                // warp that brings the last of its experts, which spreads the sums over
                // the call: summed for all 32 tokens by the last expert's they took 55 us at
                // its end.
                const int o = c.m * kTile + 4 * lane + q;
                if (o < a.H)
#pragma unroll
                    for (int x = 0; x < kRows; ++x)
                        if (x < c.rows) a.y[(int64_t)rt.order[c.row + x] * a.H + o] = sum[x];
                __syncwarp();
                int token = 0;
                bool last = false;
                __threadfence();
                if (lane < c.rows) {
                    token = rt.order[c.row + lane] / a.K;
                    last = atomicAdd(a.arrived + (c.m * 4 + q) * a.S + token, 1u) + 1 ==
                           (uint32_t)valid[token];
                }
                uint32_t ready = __ballot_sync(0xffffffffu, last);
                if (ready) __threadfence();
                while (ready) {
                    int s[kFewTokens], count = 0, from = 0;
#pragma unroll
                    for (int j = 0; j < kFewTokens; ++j) {
                        if (ready) {
                            from = __ffs(ready) - 1;
                            ready &= ready - 1;
                            ++count;
                        }
                        s[j] = __shfl_sync(0xffffffffu, token, from);
                    }
                    if (o >= a.H) continue;
                    if (count == 1)
                        few_combine<1>(a.y, weights, rt.place, a.K, a.H, o, s, 1, a.out, a.f32);
                    else
                        few_combine<kFewTokens>(a.y, weights, rt.place, a.K, a.H, o, s, count,
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

struct Shape {
    int rank;
    cuuint64_t dims[5], strides[4];   // strides of all but the innermost, in bytes
    cuuint32_t box[5];
};

cudaError_t encode(CUtensorMap *map, const void *base, bool words, const Shape &s)
{
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(
        map, words ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT8, s.rank,
        const_cast<void *>(base), s.dims, s.strides, s.box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
        words ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Parts of 64 rows of D elements as the other operand.
cudaError_t encode_rows(LayerMaps &m, const uint8_t *codes, const uint8_t *scales, int parts, int D)
{
    const cuuint64_t row = D / 2, P = parts, words = (D + 127) / 128;
    cudaError_t e = cudaSuccess;
    for (cuuint32_t i = 0; i < 2 && e == cudaSuccess; ++i)
        e = encode(&m.b[i], codes, false, {2, {row, P * kCols}, {row}, {128, kCols / 2 * (i + 1)}});
    if (e != cudaSuccess) return e;
    return encode(&m.sb, scales, true, {2, {P * 128, words}, {P * 512}, {128, 2}});
}

template <bool UP> int launch_layer(const LayerMaps &maps, LayerArgs a, cudaStream_t stream)
{
    static KernelCache kc;
    const size_t rest = 1024 + kBoxBytes + a.S * a.K * 4 + a.S * 2 +
                        Routing::bytes(a.S * a.K, a.E);
    // Two CTAs of an SM have four stages each; where the lists leave less, one CTA has
    // as many as fit.
    a.stages = (int)((kSmem - rest) / kStageBytes);
    if (a.stages < 4) a.stages = kMaxStages;
    const size_t smem = rest + (size_t)a.stages * kStageBytes;
    cudaError_t e = prepare_kernel(layer_kernel<UP>, smem, kThreads, kc, nullptr);
    if (e == cudaSuccess) {
        const int per_tile = UP ? kTile / 2 : kTile;
        const int64_t tiles_m = ((UP ? a.F : a.H) + per_tile - 1) / per_tile;
        const int64_t most = tiles_m * a.parts, room = (int64_t)sm_count() * (a.stages < kMaxStages ? 2 : 1);
        e = launch_pdl(layer_kernel<UP>, dim3((unsigned)(most < room ? most : room)),
                       dim3(kThreads), smem, stream, maps, a);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

// Parts of n entries: one for every eight of an expert and one for what is left.
int64_t most_parts(int64_t n, int64_t E) { return n < E + n / kRows ? n : E + n / kRows; }

// The workspace: x and h as eight rows, y, and the counters.
struct Places {
    int64_t x_codes, x_scales, h_codes, h_scales, y, arrived, bytes;
    Places(int64_t S, int64_t K, int64_t E, int64_t H, int64_t F)
    {
        const int64_t n = S * K, parts = most_parts(n, E);
        int64_t at = 0;
        auto take = [&](int64_t size) {
            const int64_t p = at;
            at += round_up(size, 256);
            return p;
        };
        x_codes = take(parts * kCols * H / 2);
        x_scales = take((H + 127) / 128 * parts * 512);
        h_codes = take(parts * kCols * F / 2);
        h_scales = take((F + 127) / 128 * parts * 512);
        y = take(n * H * 4);
        arrived = take((H + kTile - 1) / kTile * 4 * S * 4);
        bytes = at;
    }
};

} // namespace

size_t layer_mxfp4_workspace(int64_t S, int64_t K, int64_t E, int64_t H, int64_t F)
{
    return (size_t)Places(S, K, E, H, F).bytes;
}

int layer_mxfp4(const LayerCall &c, cudaStream_t stream)
{
    const int n = c.S * c.K;
    const Places at(c.S, c.K, c.E, c.H, c.F);
    uint8_t *ws = c.workspace;
    LayerArgs a = {};
    a.idx = c.idx;
    a.topk_w = c.topk_w;
    a.h_codes = ws + at.h_codes;
    a.h_scales = ws + at.h_scales;
    a.y = reinterpret_cast<float *>(ws + at.y);
    a.arrived = reinterpret_cast<uint32_t *>(ws + at.arrived);
    a.out = c.out;
    a.S = c.S;
    a.K = c.K;
    a.E = c.E;
    a.H = c.H;
    a.F = c.F;
    a.parts = (int)most_parts(n, c.E);
    a.f32 = c.f32;
    LayerMaps up = {}, down = {};
    const cuuint64_t E = c.E, H = c.H, F = c.F;
    const cuuint64_t up_row = H / 2, up_words = (H + 127) / 128;
    const cuuint64_t down_row = F / 2, down_words = (F + 127) / 128;
    // gates and ups as two runs of F rows
    cudaError_t e = encode(&up.a, c.up, false,
                           {5,
                            {up_row, F / 4, 2, 4, E},
                            {4 * up_row, F * up_row, up_row, 2 * F * up_row},
                            {128, 16, 2, 4, 1}});
    if (e == cudaSuccess)
        e = encode(&up.sa, c.up_scales, true,
                   {4, {F, 2, up_words, E}, {F * 4, 2 * F * 4, up_words * 2 * F * 4}, {64, 2, 2, 1}});
    if (e == cudaSuccess)
        e = encode_rows(up, ws + at.x_codes, ws + at.x_scales, a.parts, c.H);
    if (e == cudaSuccess)
        e = encode(&down.a, c.down, false,
                   {4, {down_row, H / 4, 4, E}, {4 * down_row, down_row, H * down_row}, {128, 32, 4, 1}});
    if (e == cudaSuccess)
        e = encode(&down.sa, c.down_scales, true,
                   {3, {H, down_words, E}, {H * 4, down_words * H * 4}, {kTile, 2, 1}});
    if (e == cudaSuccess)
        e = encode_rows(down, a.h_codes, a.h_scales, a.parts, c.F);
    static KernelCache kc;
    const size_t smem = Routing::bytes(n, c.E);
    if (e == cudaSuccess) e = prepare_kernel(split_kernel, smem, kThreads, kc, nullptr);
    if (e == cudaSuccess) {
        SplitArgs s = {c.x, c.idx, ws + at.x_codes, reinterpret_cast<uint32_t *>(ws + at.x_scales),
                       a.arrived, c.S, c.K, c.E, c.H, a.parts, (c.H + kTile - 1) / kTile * 4 * c.S};
        const int64_t units = (int64_t)c.S * ((c.H + 255) / 256), most = 2 * sm_count();
        const int64_t grid = (units + kThreads / 32 - 1) / (kThreads / 32);
        e = launch_pdl(split_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(kThreads),
                       smem, stream, s);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    int r = check_launch();
    if (r == MOE_OK) r = launch_layer<true>(up, a, stream);
    if (r == MOE_OK) r = launch_layer<false>(down, a, stream);
    return r;
}

// Reads and clears this file's device error bits.
cudaError_t read_layer_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_layer_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_layer_error, &zero, sizeof(uint32_t));
    return e;
}

} // namespace moe
