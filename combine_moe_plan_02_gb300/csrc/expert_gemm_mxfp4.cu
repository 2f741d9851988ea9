// The experts' product over packed rows, rows and weights in MXFP4.
//
// Bucket e is the rows off[e] .. off[e] + cnt[e] of a plan:
//   y[r, n] = sum_d x[r, d] * w[e, n, d]        r in bucket e
// with x and w E2M1 codes under E8M0 scales of 32 elements (csrc/mxfp4.cu has the
// format).  The block-scaled matrix instruction (kind::mxf4) takes codes and
// scales as they are: codes from shared memory, scales from tensor memory; sums
// are f32, for f32 outputs in parts of 4096 elements, rounded once to the output's type.
//
// Weight rows are the M side (256 TMEM lanes of a pair of CTAs), tokens the N
// side (128 or 256 columns), as in csrc/expert_gemm.cu, whose pairs, warps and
// walk over the tiles this kernel shares.  Different here:
//
// Scales.  For 128 rows and 128 elements the instruction wants 128 words (four
// scale bytes each) as 32 lanes x 4 columns, row 32 j + q in column j of lane q.
// A copy from shared memory to tensor memory (tcgen05.cp, 32x128b) puts the four
// words of 16 bytes side by side in one lane, so 128 neighbouring words of the
// scale array arrive as row 4 q + j in column j of lane q.  The codes are made to
// match: TMA reads a tensor of rows as [4][rows / 4] and so lays row 4 q + j in
// row 32 j + q of the stage.  Nothing is rearranged by a thread.  A copy begins on
// 16 bytes, four words: tiles begin at a row that is a multiple of 4, up to three
// rows before their bucket; those columns are not stored (columns are
// independent).  Rows of a tensor are a multiple of 4.
//
// Tensor memory.  Two accumulators of 256 columns would leave no room for scales.
// They overlap by 128 columns (0 .. 255 and 128 .. 383): the storing warps take the
// shared columns into registers first and hand them on, so the next tile waits for
// half of the reads and no store.  The rest holds the scales of each stage's block, so
// that a stage's copy into it, which begins when the products that read the stage before
// are done, frees its columns too.
//
// Output.  Lane 32 j + q of the accumulator is output 4 q + j: the four warps that
// read its quarters meet in shared memory, and whole output rows leave in 16-byte
// stores, just those of the bucket.
//
// What bounds it, 64 buckets of 512 rows, 7168 -> 4096, bf16 out: 291 us (6.6 PFLOP/s; 68 %
// of the tensor pipe's cycles) with 17.5 TB/s of operands from L2; without the token
// operand's copies 270, without the stores 265, without the copies of scales 277, with
// half of the products 265 us.  Buckets of 512 rows on average: 321 us, as columns come
// in 128s; for seconds on end the power limit makes that 366 to 379.  2048 -> 7168: 197 us,
// stores (470 MB) and operands.  4 rows in each of 256 buckets, 6144 -> 4096: 323 us (7.0
// TB/s of weights with 128 tokens of 8 experts, 480 us).

#include "pair.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kStoreWarps = 8;      // two for each quarter of the lanes
constexpr int kThreads = 128 + 32 * kStoreWarps;
constexpr int kLanes = 128;         // TMEM lanes of a CTA: outputs
constexpr int kM = 2 * kLanes;      // of the pair
constexpr int kN = 256;             // columns of a tile, or half as many
constexpr int kK = 256;             // elements of a reduction block: 128 bytes of codes
constexpr int kABytes = kLanes * kK / 2;
constexpr int kScaleWords = 2;      // words of scales in a block and row
constexpr int kSABytes = kLanes * kScaleWords * 4;
constexpr int kStageBytes = 2 * kABytes + 3 * kSABytes;
constexpr int kStages = 5;
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kMaxStages = 6;       // of 128 columns
constexpr int kAccTwo = 128;        // first column of the second accumulator
constexpr int kScaleAt = 384;       // first column of the scales
constexpr int kScaleCols = 24;      // of a block: 2 x (4 + 8)
constexpr int kTmemCols = 512;
constexpr int64_t kLongest = 32768;
// Blocks of an accumulator of f32 outputs, 64 steps.  Sums lose nothing while all terms lie
// within 24 bits of the largest sum; where a row's scales are spread further each step of 64
// elements cuts low bits off.  Scales of 2^10 and 2^20 leave 2.9e-7 and 1.3e-6 of the result
// (2-norm, 32768 elements; plain f32 sums 2.0e-7 and 3.7e-7; one accumulator 2.9e-6 and
// 1.0e-5).  A part costs 0.3 us of a pair, in which the accumulators' shared columns are
// read: 32768 x 7168 -> 4096 takes 370 us with two parts, 362 with one, 395 with four.
constexpr int kPart = 16;

__device__ uint32_t g_mxgemm_error;  // kErrExpertTimeout | kErrExpertBucket

struct MxArgs {
    const int32_t *cnt;   // [E]
    const int64_t *off;   // [E + 1]
    int64_t rows;
    int E;
    int M;                // outputs of a row
    int K;                // reduction length
    uint8_t *out;         // [rows, M]
};

// The maps of the operands: codes of the weights and of the rows (256 columns,
// then boxes of 8, 16, 24, 32 rows of a quarter), scales likewise.
struct MxMaps {
    CUtensorMap a, sa, b, sb[2], part[4];
};

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t scale_a, uint32_t scale_b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"((uint32_t)add)
        : "memory");
}

// 512 bytes of both CTAs' shared memory to 4 columns of both, for each quarter of
// the lanes.
__device__ __forceinline__ void copy_scales(uint32_t d, uint64_t src)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(src) : "memory");
}

// Codes in shared memory: rows of 128 bytes along the reduction, 128-byte swizzle.
__device__ __forceinline__ uint64_t code_desc(uint32_t addr)
{
    return ((uint64_t)(addr & 0x3ffff) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Scales in shared memory: rows of 16 bytes one after another, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)
{
    return ((uint64_t)(addr & 0x3ffff) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) |
           (1ull << 46);
}

// E2M1 operands, E8M0 scales; `half`: which two of a word's four scales.
__device__ __forceinline__ uint32_t instr_desc(int n, int half)
{
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           (1u << 23) | ((uint32_t)(kM >> 4) << 24) | ((uint32_t)(2 * half) << 29);
}

__device__ __forceinline__ void tma_4d(void *dst, const CUtensorMap *map, uint32_t bar, int x,
                                       int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// --- tiles -------------------------------------------------------------------

struct Tile {
    int e, m0;
    int n0;       // row of the first column, a multiple of 4
    int cols;     // columns: 128 or 256
    int from;     // columns that are stored: from .. to
    int to;
};

struct Schedule {
    int *start;   // [E + 1] first tile of each bucket
    int *first;   // [E] first row
    int *fill;    // [E] rows
    int widest;   // columns of the largest bucket
    int cursor;   // bucket of the last tile asked for; tiles are asked for in order
};

__device__ __forceinline__ Tile tile_of(const MxArgs &a, Schedule &s, int t)
{
    // the last bucket that begins at or before t
    int past = s.cursor + 4;
    while (s.cursor < past && t >= s.start[s.cursor + 1]) ++s.cursor;
    if (t >= s.start[s.cursor + 1]) {
        past = a.E;
        while (past - s.cursor > 1) {
            const int mid = (s.cursor + past) >> 1;
            if (s.start[mid] <= t) s.cursor = mid;
            else past = mid;
        }
    }
    Tile r;
    r.e = s.cursor;
    const int local = t - s.start[r.e], row = s.first[r.e], shift = row & 3;
    const int end = shift + s.fill[r.e], parts = ceil_div(end, kN);
    const int m = local / parts, i = local - m * parts;
    r.m0 = m * kM;
    r.n0 = row - shift + i * kN;
    r.from = i ? 0 : shift;
    r.to = min(kN, end - i * kN);
    r.cols = r.to > kN / 2 ? kN : kN / 2;
    return r;
}

// Lists the tiles: every thread of the CTA takes part.
__device__ void build_schedule(const MxArgs &a, Schedule &s)
{
    __shared__ int s_warp[kThreads / 32], s_most[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mt = ceil_div(a.M, kM);
    int base = 0, most = 0;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + tid;
        int tiles = 0;
        if (e < a.E) {
            int64_t f = __ldg(a.off + e), c = __ldg(a.cnt + e);
            if (f < 0 || c < 0 || f > a.rows - c) {  // f + c may not fit
                // never outside the rows: the bucket is left out and reported
                atomicOr(&g_mxgemm_error, kErrExpertBucket);
                f = c = 0;
            }
            s.first[e] = (int)f;
            s.fill[e] = (int)c;
            const int end = (int)(f & 3) + (int)c;
            if (c) {
                most = max(most, end);
                tiles = mt * ceil_div(end, kN);
            }
        }
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        int before = base, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
        if (e < a.E) s.start[e + 1] = before + sum;
        base += total;
        __syncthreads();
    }
    if (tid == 0) s.start[0] = 0;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_most[warp] = most;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) s.widest = max(s.widest, s_most[w]);
}

// --- the kernel ----------------------------------------------------------------

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_free, drain;
    uint32_t tmem;
    volatile int stop;
};

// Where the four quarters of a block of 32 columns meet: 32 tokens, for each the
// outputs of the quarters one after another.  Rows of bf16 are 64 bytes apart
// beyond their 256, so that two of them can be read at once.
template <typename Tout> struct Meet {
    static constexpr int kQuarter = 32 * (int)sizeof(Tout);
    static constexpr int kRow = 4 * kQuarter + (sizeof(Tout) == 2 ? 64 : 0);
    static constexpr int kBytes = 32 * kRow;
};

// SUMS: f32 outputs of more than one part.
template <typename Tout, bool SUMS>
__global__ void __launch_bounds__(kThreads, 1)
mxgemm_kernel(const __grid_constant__ MxMaps maps, MxArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    uint8_t *meet = ring + kRingBytes;
    int *lists = reinterpret_cast<int *>(meet + 2 * Meet<Tout>::kBytes);
    Schedule sched = {lists, lists + a.E + 1, lists + 2 * a.E + 1, 0, 0};
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh.full[i], 4);   // both operands of both CTAs
            mbar_init(&sh.empty[i], 1);
        }
        mbar_init(&sh.acc_full[0], 1);
        mbar_init(&sh.acc_full[1], 1);
        mbar_init(&sh.acc_free, 2 * kStoreWarps);  // the storing warps of both CTAs
        mbar_init(&sh.drain, 1);
        sh.stop = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&sh.tmem, kTmemCols);
    griddep_wait();  // the plan and the operands come from earlier stream work
    griddep_launch_dependents();
    build_schedule(a, sched);        // ends with a CTA barrier
    cluster_sync();                  // both CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int tiles = sched.start[a.E];
    // Five stages of 128 + 128 rows, or six where no tile is wider than 128 columns.
    const bool narrow = sched.widest <= kN / 2;
    const int rows_b = narrow ? kN / 4 : kN / 2;
    const int scales_at = kABytes + rows_b * 128;  // the weights', then the rows'
    const int stage_bytes = scales_at + kSABytes + (narrow ? 1 : 2) * kSABytes;
    const int stages = narrow ? kMaxStages : kStages;
    const int blocks = ceil_div(a.K, kK);

    // Of several parts a storing thread holds up to 128 sums.  The block starts with 384 x
    // 168 = 64512 registers, which 128 x 72 + 256 x 216 are too.
    if (warp < 4) {
        if (SUMS) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 || warp == 2) {
            const bool weights = warp == 0;
            if (elect_one()) {
                const uint32_t full = addr_in(sh.full, 0);
                Ring r(stages);
                int64_t j = 0;  // blocks copied
                bool ok = true;
                for (int t = pair; t < tiles && ok; t += pairs) {
                    const Tile c = tile_of(a, sched, t);
                    const bool wide = c.cols == kN;
                    const int eights = ceil_div(c.to, 32);  // rows of a quarter, in eights
                    const uint32_t bytes = weights ? kABytes + kSABytes
                                           : wide  ? kABytes + 2 * kSABytes
                                                   : eights * 2048 + kSABytes;
                    for (int b = 0; b < blocks; ++b, ++j) {
                        if (j >= stages && !wait(&sh.empty[r.at], r.round ^ 1, &sh.stop)) {
                            ok = false;
                            break;
                        }
                        uint8_t *stage = ring + r.at * stage_bytes;
                        uint8_t *scales = stage + scales_at;
                        const uint32_t bar = full + r.at * 8;
                        arrive_expect_at(bar, bytes);
                        if (weights) {
                            const int m = c.m0 + rank * kLanes;
                            tma_4d(stage, &maps.a, bar, b * 128, m / 4, 0, c.e);
                            tma_3d(scales, &maps.sa, bar, m, 2 * b, c.e);
                        } else {
                            uint8_t *codes = stage + kABytes;
                            if (wide) {
                                tma_3d(codes, &maps.b, bar, b * 128, c.n0 / 4 + rank * 32, 0);
                            } else {
                                // columns 64 rank ..: quarters 2 rank and 2 rank + 1
                                const CUtensorMap *map = &maps.part[eights - 1];
                                for (int i = 0; i < 2; ++i)
                                    tma_3d(codes + i * 4096, map, bar, b * 128, c.n0 / 4,
                                           2 * rank + i);
                            }
                            tma_2d(scales + kSABytes, &maps.sb[wide], bar, c.n0, 2 * b);
                        }
                        r.next();
                    }
                }
                if (!ok && rank == 0) {
                    // leave no copy in flight: both CTAs' copies arrive here
                    for (int64_t i = j > stages ? j - stages : 0; i < j; ++i)
                        (void)wait_slow(&sh.full[i % stages], (uint32_t)(i / stages) & 1, nullptr);
                }
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // One thread does it all: what it issues in a block (two waits, up to six
            // copies of scales, four products) is close to what bounds the kernel.
            if (elect_one()) {
                Ring r(stages);
                int i = 0;  // accumulators begun
                bool ok = true;
                const uint32_t scale_cols = narrow ? 16 : kScaleCols;
                for (int t = pair; t < tiles && ok; t += pairs) {
                    const Tile c = tile_of(a, sched, t);
                    uint32_t acc = 0;
                    int next = 0;  // first block of the next accumulator
                    const uint32_t low = instr_desc(c.cols, 0), high = instr_desc(c.cols, 1);
                    const bool wide = c.cols == kN;
                    for (int b = 0; b < blocks; ++b) {
                        const bool fresh = b == next;
                        if (fresh) {
                            next = SUMS ? next + kPart : blocks;
                            if (SUMS && b > 0) mma_commit(&sh.acc_full[(i - 1) & 1], 0);
                            // the columns that this accumulator shares with the one before
                            // have been read, and all of the one before that
                            if (i > 0 && !wait(&sh.acc_free, (uint32_t)(i - 1) & 1, &sh.stop)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            acc = tmem + (i & 1) * kAccTwo;
                            ++i;
                        }
                        if (!wait(&sh.full[r.at], r.round, &sh.stop)) {
                            ok = false;
                            break;
                        }
                        const uint32_t stage = smem_u32(ring) + r.at * stage_bytes;
                        tc_fence_after();
                        const uint32_t sa = tmem + kScaleAt + (uint32_t)r.at * scale_cols;
                        const uint32_t sb = sa + 8;
                        const uint64_t from_a = scale_desc(stage + scales_at);
                        const uint64_t from_b = from_a + (kSABytes >> 4);
                        const uint64_t da = code_desc(stage), db = da + (kABytes >> 4);
                        const int left = a.K - b * kK;  // 64 elements a product
                        copy_scales(sa, from_a);
                        copy_scales(sb, from_b);
                        if (wide) copy_scales(sb + 4, from_b + 32);
                        mma_mxf4(acc, da, db, low, sa, sb, !fresh);
                        if (left > 64) mma_mxf4(acc, da + 2, db + 2, high, sa, sb, true);
                        if (left > 128) {
                            const uint32_t sa1 = sa + 4, sb1 = sb + (wide ? 8 : 4);
                            copy_scales(sa1, from_a + 32);
                            copy_scales(sb1, from_b + (c.cols >> 2));
                            if (wide) copy_scales(sb1 + 4, from_b + 96);
                            mma_mxf4(acc, da + 4, db + 4, low, sa1, sb1, true);
                            if (left > 192) mma_mxf4(acc, da + 6, db + 6, high, sa1, sb1, true);
                        }
                        mma_commit(&sh.empty[r.at], 0);
                        r.next();
                    }
                    if (ok) mma_commit(&sh.acc_full[(i - 1) & 1], 0);
                }
                mma_commit(&sh.drain, 0);  // nothing is issued after this
            }
            __syncwarp();
        } else if (warp == 3) {
            zero_gaps(a.out, (int64_t)a.M * (int)sizeof(Tout), a.rows, a.cnt, a.off, a.E,
                      blockIdx.x, gridDim.x);
        }
        __syncwarp();
    } else {
        if (SUMS) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        using Me = Meet<Tout>;
        const int q = warp & 3;             // this warp's quarter of the lanes
        const int odd = warp >> 2 & 1;      // its blocks of 32 columns: even or odd ones
        uint8_t *box = meet + odd * Me::kBytes;
        auto join = [&] {
            asm volatile("bar.sync %0, %1;" ::"r"(1 + odd), "n"(128) : "memory");
        };
        // whether all four warps go on: one that gave up must not leave the others
        // at their next meeting.  Lanes may leave a wait apart, and meet as whole warps.
        auto agree = [&](bool ok) {
            uint32_t all;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\t"
                         "setp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, %2, %3, p;\n\t"
                         "selp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"((uint32_t)ok), "r"(1 + odd), "n"(128)
                         : "memory");
            return all != 0;
        };
        const uint32_t free_at = addr_in(&sh.acc_free, 0);
        const int parts = ceil_div(blocks, kPart);  // of a tile's reduction
        int i = 0;
        for (int t = pair; t < tiles; t += pairs) {
            const Tile c = tile_of(a, sched, t);
            const int count = c.cols / 64, used = ceil_div(c.to, 4);
            const int m = c.m0 + rank * kLanes;
            // what the next tile or part needs of this accumulator is in registers
            auto hand_on = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(free_at);
            };
            auto store = [&](int jj, const uint32_t(&v)[32]) {
                const int before = (jj >> 2) * 128 + (jj & 3);  // token of x: before + 4 x
                join();  // what was here has been read
                uint8_t *mine = box + q * Me::kQuarter + lane * (int)sizeof(Tout);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    if (x >= used) break;
                    const float f = __uint_as_float(v[x]);
                    if (sizeof(Tout) == 2)
                        *reinterpret_cast<__nv_bfloat16 *>(mine + x * Me::kRow) =
                            __float2bfloat16_rn(f);
                    else
                        *reinterpret_cast<float *>(mine + x * Me::kRow) = f;
                }
                join();
                constexpr int kAcross = 128 * (int)sizeof(Tout) / 16;  // lanes of a row
                const int at = lane % kAcross;
                const int first = m + at * (16 / (int)sizeof(Tout));   // its outputs
#pragma unroll
                for (int x0 = 0; x0 < 8; x0 += 32 / kAcross) {
                    const int x = q * 8 + x0 + lane / kAcross;
                    const int token = before + 4 * x;
                    if (token < c.from || token >= c.to || first >= a.M) continue;
                    const uint8_t *p = box + x * Me::kRow + at * 4;
                    uint32_t w[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        w[h] = *reinterpret_cast<const uint32_t *>(p + h * Me::kQuarter);
                    // bf16: outputs 8 at .. of four quarters, two of each in a word
                    const uint4 o = sizeof(Tout) == 2
                                        ? make_uint4(__byte_perm(w[0], w[1], 0x5410),
                                                     __byte_perm(w[2], w[3], 0x5410),
                                                     __byte_perm(w[0], w[1], 0x7632),
                                                     __byte_perm(w[2], w[3], 0x7632))
                                        : make_uint4(w[0], w[1], w[2], w[3]);
                    st16(a.out + ((int64_t)(c.n0 + token) * a.M + first) * (int)sizeof(Tout), o);
                }
            };
            // This warp's blocks, the columns that the accumulators share first: the last
            // ones of accumulator 0, the first ones of accumulator 1.
            if (SUMS) {
                uint32_t sum[kN / 64][32];  // f32
#pragma unroll
                for (int k = 0; k < kN / 64; ++k)
#pragma unroll
                    for (int x = 0; x < 32; ++x) sum[k][x] = 0;
                bool ok = true;
                for (int p = 0; p < parts; ++p, ++i) {
                    const int buf = i & 1;
                    ok = wait_warp(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccTwo + odd * 32;
                    // two blocks, half of one added while the next half is read
                    auto take = [&](int k, int l) {
                        uint32_t v[2][16];
                        tmem_load(acc + k * 64, v[0]);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            tmem_wait(v[h & 1]);
                            if (h < 3)
                                tmem_load(acc + (h < 1 ? k : l) * 64 + (h + 1) % 2 * 16, v[(h + 1) & 1]);
                            uint32_t *to = sum[h < 2 ? k : l] + h % 2 * 16;
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                to[x] = __float_as_uint(__uint_as_float(to[x]) +
                                                        __uint_as_float(v[h & 1][x]));
                        }
                    };
                    if (buf == 0 && count == 4) {
                        take(3, 2);
                        hand_on();
                        take(1, 0);
                    } else {
                        take(0, 1);
                        hand_on();
                        if (count == 4) take(2, 3);
                    }
                }
                if (!agree(ok)) break;
#pragma unroll
                for (int k = 0; k < kN / 64; ++k)
                    if (k < count) store(2 * k + odd, sum[k]);
            } else {
                const int buf = i & 1;
                if (!agree(wait(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop))) break;
                tc_fence_after();
                ++i;
                const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccTwo;
                // The first two are read before anything is stored; that covers what is
                // shared.
                auto block = [&](int k) { return 2 * (buf ? k : count - 1 - k) + odd; };
                uint32_t two[2][32];
                tmem_load(acc + block(0) * 32, two[0]);
                tmem_load(acc + block(1) * 32, two[1]);
                tmem_wait(two[0]);
                tmem_wait(two[1]);
                hand_on();
                store(block(0), two[0]);
                store(block(1), two[1]);
                for (int k = 2; k < count; ++k) {
                    tmem_load(acc + block(k) * 32, two[0]);
                    tmem_wait(two[0]);
                    store(block(k), two[0]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) (void)wait_slow(&sh.drain, 0, nullptr);  // the last matrix instruction
    __syncwarp();
    cluster_sync();  // no arrival or product of the other CTA is under way
    if (tid == 0 && sh.stop) atomicOr(&g_mxgemm_error, kErrExpertTimeout);
    if (warp == 1) tmem_free(tmem, kTmemCols);
}

// --- host ----------------------------------------------------------------------

// A map over dims (innermost first); strides in bytes of all but the first.
cudaError_t encode(CUtensorMap *map, const void *base, bool words, int rank,
                   const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box)
{
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = fn(
        map, words ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
        const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
        words ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename Tout, bool SUMS = false>
int launch_mx(const MxMaps &maps, const MxArgs &a, int clusters, cudaStream_t stream)
{
    static KernelCache kc;
    auto kernel = mxgemm_kernel<Tout, SUMS>;
    const size_t smem =
        1024 + kRingBytes + 2 * Meet<Tout>::kBytes + (3 * (size_t)a.E + 1) * sizeof(int);
    cudaError_t e = prepare_kernel(kernel, smem, kThreads, kc, nullptr);
    if (e == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = MOE_USE_PDL;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * clusters);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kernel, maps, a);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    return check_launch();
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT int moe_expert_gemm_mxfp4(const uint8_t *x_codes, const uint8_t *x_scales, int64_t rows,
                                     const uint8_t *w_codes, const uint8_t *w_scales, int64_t N,
                                     int64_t D, int E, const int32_t *cnt, const int64_t *off,
                                     void *y, int y_dtype, moe_stream_t stream)
{
    MOE_TRACE("moe_expert_gemm_mxfp4");
    if (y_dtype != MOE_BF16 && y_dtype != MOE_F32) return MOE_EINVAL;
    if (rows < 0 || rows >= ((int64_t)1 << 31) || E < 1 || E > 1024) return MOE_EINVAL;
    if (N < 1 || N >= (1 << 24) || D < 1 || D > kLongest) return MOE_EINVAL;
    if (rows == 0) return MOE_OK;  // no rows, no output
    if (!x_codes || !x_scales || !w_codes || !w_scales || !cnt || !off || !y) return MOE_EINVAL;
    const int64_t mt = (N + kM - 1) / kM;
    if (E * mt * (rows / kN + 2) >= ((int64_t)1 << 31)) return MOE_EINVAL;
    if (rows % 4 || N % 8 || D % 32 || !aligned16(x_codes) || !aligned16(x_scales) ||
        !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y))
        return MOE_EALIGN;
    MxArgs a = {cnt, off, rows, E, (int)N, (int)D, static_cast<uint8_t *>(y)};
    MxMaps maps = {};
    const cuuint64_t row = (cuuint64_t)D / 2, words = (cuuint64_t)(D + 127) / 128;
    const cuuint64_t R = (cuuint64_t)rows, n = (cuuint64_t)N;
    cudaError_t e = cudaSuccess;
    auto make = [&](CUtensorMap *map, const void *base, bool w, int rank, const cuuint64_t *dims,
                    const cuuint64_t *strides, const cuuint32_t *box) {
        if (e == cudaSuccess) e = encode(map, base, w, rank, dims, strides, box);
    };
    {
        const cuuint64_t dims[4] = {row, n / 4, 4, (cuuint64_t)E};
        const cuuint64_t strides[3] = {4 * row, row, n * row};
        const cuuint32_t box[4] = {128, 32, 4, 1};
        make(&maps.a, w_codes, false, 4, dims, strides, box);
    }
    {
        const cuuint64_t dims[3] = {n, words, (cuuint64_t)E};
        const cuuint64_t strides[2] = {n * 4, words * n * 4};
        const cuuint32_t box[3] = {kLanes, kScaleWords, 1};
        make(&maps.sa, w_scales, true, 3, dims, strides, box);
    }
    {
        const cuuint64_t dims[3] = {row, R / 4, 4};
        const cuuint64_t strides[2] = {4 * row, row};
        const cuuint32_t box[3] = {128, 32, 4};
        make(&maps.b, x_codes, false, 3, dims, strides, box);
        for (cuuint32_t i = 0; i < 4; ++i) {
            const cuuint32_t quarter[3] = {128, 8 * (i + 1), 1};
            make(&maps.part[i], x_codes, false, 3, dims, strides, quarter);
        }
    }
    for (cuuint32_t i = 0; i < 2; ++i) {
        const cuuint64_t dims[2] = {R, words};
        const cuuint64_t strides[1] = {R * 4};
        const cuuint32_t box[2] = {128 * (i + 1), kScaleWords};
        make(&maps.sb[i], x_scales, true, 2, dims, strides, box);
    }
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    const int64_t most = mt * (rows / kN + 2 * (rows < E ? rows : E));
    const int pairs = sm_count() / 2;
    const int clusters = (int)(most < pairs ? most : pairs);
    // A kernel of its own for one part: it starts with fewer registers (108 rows over 128
    // experts' buckets of 4, 1344 -> 2128: 0.5 us of 26).
    const bool sums = D > (int64_t)kPart * kK;
    if (y_dtype != MOE_F32)
        return launch_mx<__nv_bfloat16>(maps, a, clusters, (cudaStream_t)stream);
    return sums ? launch_mx<float, true>(maps, a, clusters, (cudaStream_t)stream)
                : launch_mx<float>(maps, a, clusters, (cudaStream_t)stream);
}

namespace moe {
// Reads and clears this file's device error bits.
cudaError_t read_mxgemm_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_mxgemm_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_mxgemm_error, &zero, sizeof(uint32_t));
    return e;
}
} // namespace moe
