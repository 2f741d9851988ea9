// The experts' products over packed rows, and their gradients.
//
// Bucket e is the rows off[e] .. off[e] + cnt[e] of a plan.  With w [E, N, D]:
//   forward   y[r, n]    = sum_d x[r, d] * w[e, n, d]          r in bucket e
//   rows'     dx[r, d]   = sum_n dy[r, n] * w[e, n, d]
//   weights'  dw[e, n, d] = sum_{r in e} dy[r, n] * x[r, d]
// bf16 operands, f32 sums (tensor memory), one rounding to the output's type.
//
// One tcgen05 kernel does all three.  The M side of the matrix instruction
// (256 TMEM lanes of a pair of CTAs) is always the dimension that is
// contiguous in the output: weight rows n (forward), d (the gradients).  The N
// side (up to 256 TMEM columns) is the tokens of one bucket, or the rows n of
// dw.  A bucket of c tokens is cut into ceil(c / 256) parts of nearly equal
// numbers of 32-column steps, so a bucket costs at most 31 idle columns and one
// token costs 32 columns instead of a padded tile of rows.  Rows of other
// buckets that a copied box holds land in columns that are never stored;
// columns are independent, so nothing they hold (NaN included) matters.  The
// weights' gradient reduces over the tokens: of a bucket's last block just the
// bucket's rows are copied, and zeros after them up to a multiple of 16 rows.
//
// Two CTAs on neighbouring SMs work on one tile of 256 x 256 (cta_group::2):
// each holds its 128 lanes of the M side and half of the N side in shared
// memory, so a pair reads 64 KB per block of 64 along the reduction where two
// single CTAs of 128 x 256 read 96 KB.
//
// Where a call of few rows has fewer tiles than half of the pairs, two or four
// pairs of a cluster share a tile's reduction; the first adds the others' sums,
// which they write into its shared memory, in a fixed order.  Otherwise:
//
// A pair is persistent (one per two SMs) and walks the tiles of all buckets,
// which it lists itself from cnt and off: the sizes stay on the device.  Warps
// 0 and 2 copy the operands' blocks of 64 along the reduction with TMA into a
// ring of stages (one warp each: issuing a copy takes 60 to 100 cycles and a
// wait and an arrival as much again, against 512 cycles of products a block),
// warp 1 of the first CTA issues the matrix instructions, warp 3 clears the
// rows of the output that belong to no bucket, warps 4 to 11 store.  Two accumulators of 256
// columns let the stores of a tile overlap the next tile's products.  Every
// wait is bounded.
//
// What bounds it, 64 buckets of 512 rows, 2048 x 7168, bf16 out: 549 us forward,
// 550 us for the rows (1753, 1749 TFLOP/s; 87 % of the tensor pipe's cycles),
// the copies from L2: six stages of 32 KB are what fits, with four it takes 618
// us, without the tokens' copies 499 us.  For seconds on end the power limit
// sets the pace: 620 to 640 us.  Buckets of 512 rows on average, half of them
// cut into three parts: 590 us (670 to 690 us for seconds).  The weights'
// gradient: 606 us in bf16 (1588 TFLOP/s), 767 us in f32, where 4.36 GB move and products, copies
// and stores share L2 and shared memory.  One row in each of 8 buckets, 2048 x
// 6144: 35 us, the weights at 6.5 TB/s behind 4 us of launch and tile list; 1024
// rows in 256 buckets: 885 us (7.3 TB/s).  64 pairs' work taken over by cluster
// launch control instead of the fixed walk measured 1 % slower, tiles of 512
// columns 33 % (the next tile waits for both accumulators' stores).

#include "pair.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kStoreWarps = 8;      // two for each quarter of the lanes
constexpr int kThreads = 128 + 32 * kStoreWarps;
constexpr int kLanes = 128;         // TMEM lanes of a CTA: outputs along the contiguous dimension
constexpr int kM = 2 * kLanes;      // of the pair
constexpr int kN = 256;             // TMEM columns of one accumulator
constexpr int kK = 64;              // reduction block: 128 bytes of bf16
constexpr int kStep = 32;           // columns come in these steps, half of them from each CTA
constexpr int kABytes = kLanes * kK * 2;
constexpr int kBBytes = kN / 2 * kK * 2;
constexpr int kRingBytes = 6 * (kABytes + kBBytes);
constexpr int kMaxStages = 10;
constexpr int kBoxArea = 2048;      // of each storing warp
constexpr int kSplitRows = 64;      // rows of a call whose reductions may be split
constexpr int kSplitBytes = kSplitRows * kLanes * 4;  // one pair's sums, in each CTA

__device__ uint32_t g_expert_error;  // kErrExpertTimeout | kErrExpertBucket

enum Mode { kForward = 0, kRowGrad = 1, kWeightGrad = 2 };

struct ExpertArgs {
    const int32_t *cnt;   // [E]
    const int64_t *off;   // [E + 1]
    int64_t rows;
    int E;
    int M;                // contiguous output dimension
    int N;                // rows of a weight (weights' gradient)
    int K;                // reduction length (the other two)
    int split;            // pairs that share a tile's reduction
    uint8_t *out;
};

// Stored boxes: 32 outputs wide, kRows columns of the accumulator high, each
// storing warp with room for kTurns of them.  The weights' gradient has few
// products for each output and is often bound by these stores, where a box
// costs its fixed part: 256 buckets of 33 rows, 1024 x 2048, in bf16 take 186 us
// in boxes of 32 rows and 250 us in 16; 64 ragged buckets of 512, 2048 x 7168,
// in f32 780 us in boxes of 16, 798 us in two of 8 and 1114 us in four of 4.
// Where rows are columns, a box holds whole columns of one bucket and the rest
// leaves row by row: 16.
//
// JOIN = 4 puts the four quarters of the lanes into one box, for a large bf16
// weights' gradient whose rows are not a multiple of 32 bytes: every row of a
// box then begins and ends inside a sector, and a sector written in parts costs
// most where the output does not stay in L2.  128 buckets of 62 rows, 1904 x
// 6952 (3.4 GB): 729 us, and 1186 us in boxes of one warp; 512 x 2952 (387 MB):
// 96 and 113 us; 344 x 2952 (260 MB): 75 and 68 us.  Where rows are whole
// sectors one warp's boxes cost less: 1904 x 6976, 693 and 611 us.
template <int MODE, typename Tout, int JOIN> struct Boxes {
    static constexpr int kRows = MODE == kWeightGrad && sizeof(Tout) == 2 ? 32 : 16;
    static constexpr int kWidth = 32 * JOIN;
    static constexpr int kBytes = kRows * kWidth * (int)sizeof(Tout);
    static constexpr int kTurns = JOIN * kBoxArea / kBytes;
};

// --- tcgen05 ---------------------------------------------------------------

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle.  Rows along the
// reduction (K-major): 8 rows of 128 bytes are 1024 bytes, the next 8 follow.
// Across it (MN-major): 64 outputs are one 128-byte row, 8 reduction steps are
// 1024 bytes and the next 64 outputs start kK rows (8192 bytes) further on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn_major)
{
    const uint64_t lead = mn_major ? (kK * 128) >> 4 : 1;
    return ((uint64_t)(addr & 0x3ffff) >> 4) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: f32 accumulator, bf16 operands.
__device__ __forceinline__ uint32_t instr_desc(int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}

// Rows y .. y + len of 64 columns, in boxes of rows inside their tensor, one for
// each digit of len to base 4 (`maps`: of 48, 32, 16, 12, 8, 4, 3, 2, 1 rows), and
// zeros up to a multiple of 16 rows at least: a box of 16, or where that would
// pass the block's 64 rows one or two that end with it (`zeros`: of 16, 8, .. 1
// rows).  So a last block arrives like any other: no thread clears rows that the
// other CTA's matrix instruction reads, which would have to be released at
// cluster scope (0.8 us a block).  The swizzle goes by the address in shared
// memory, so a box may begin at any row.  64 buckets of 512 rows on average, 2048 x
// 7168: 793 us in f32, 628 in bf16; of 512 each, without such blocks, 765 and 603;
// with one box for each bit of len 806 and 662, of the rows of zeros too.
__device__ __forceinline__ void tma_tail(uint8_t *dst, const CUtensorMap *maps,
                                         const CUtensorMap *zeros, uint32_t bar, int x, int y,
                                         int len)
{
#pragma unroll
    for (int s = 4; s >= 0; s -= 2, maps += 3) {
        const int digit = len >> s & 3;
        if (digit) {
            tma_2d(dst, maps + 3 - digit, bar, x, y);
            dst += (digit << s) * 128;
            y += digit << s;
        }
    }
    int h = 16;
    while (h > kK - len) {
        h >>= 1;
        ++zeros;
    }
    tma_2d(dst, zeros, bar, 0, 0);
    if (len + h < kK && len > kK - 16)
        tma_2d(dst + (kK - len - h) * 128, zeros, bar, 0, 0);
}

// What it copies, in rows.
__device__ __forceinline__ int tail_rows(int len)
{
    const int pad = kK - len;
    if (pad >= 16) return len + 16;
    const int h = 1 << (31 - __clz(pad));
    return len + (pad == h ? h : 2 * h);
}

// A box from this CTA's shared memory to global memory; what lies outside the
// tensor is not written.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int x, int y,
                                          int z, bool depth)
{
    if (depth)
        asm volatile(
            "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
            ::"l"(map), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                map),
            "r"(smem_u32(src)), "r"(x), "r"(y)
            : "memory");
}

// Parts of a tile's reduction that have an accumulator each.  The tensor core
// cuts a sum's low bits off at every step of 16, which after 1048 products
// leaves a relative error of 1e-6 in the 2-norm and grows with their number.
// For f32 outputs at most 12 blocks (768 products) are summed there; the
// storing warps add the parts in registers, rounding to nearest.  The bf16
// outputs are rounded 1000 times more coarsely: up to 32768 products take one
// accumulator, which loses 2.4e-4 of a sum at most where the rounding is up to
// 3.9e-3.  2^23 positive products come out 1 to 5 % low that way, so calls whose
// reductions may be longer run a LONG kernel with parts of 128 blocks.  Such a
// part takes 35 us, and its sums wait in local memory for the next.  The code
// for it costs the others 1 to 5 % (64 ragged buckets of 512, 2048 x 7168, rows'
// gradient 603 and 619 us, weights' gradient 631 and 647 us), hence a kernel of
// its own.
constexpr int64_t kLongest = 32768;

template <typename Tout, bool LONG> __device__ __forceinline__ int reduction_parts(int blocks)
{
    constexpr int kPartBlocks = sizeof(Tout) == 4 ? 12 : 128;
    return sizeof(Tout) == 4 || LONG ? max(1, (blocks + kPartBlocks - 1) / kPartBlocks) : 1;
}

// --- tiles -------------------------------------------------------------------

struct Tile {
    int e, m0;
    int n0;       // first column: a row of the packed rows, or a row of dw[e]
    int n;        // columns that are stored
    int from;     // first reduction block
    int blocks;   // reduction blocks
    int last;     // reduction length of the last block (1..64)
    int row;      // first row of the bucket (weights' gradient)
};

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The tiles of all buckets, in shared memory.
struct Schedule {
    int *start;   // [E + 1] first tile of each bucket
    int *first;   // [E] first row
    int *fill;    // [E] rows
    int widest;   // rows of the largest bucket
    int cursor;   // bucket of the last tile asked for; tiles are asked for in order
};

template <int MODE>
__device__ __forceinline__ int bucket_tiles(const ExpertArgs &a, int fill)
{
    const int mt = ceil_div(a.M, kM);
    return MODE == kWeightGrad ? mt * ceil_div(a.N, kN) : mt * ceil_div(fill, kN);
}

template <int MODE> __device__ __forceinline__ Tile tile_of(const ExpertArgs &a, Schedule &s, int t)
{
    Tile r;
    if (MODE == kWeightGrad) {
        r.e = t / bucket_tiles<MODE>(a, 0);  // every bucket has as many
    } else {
        // the last bucket that begins at or before t: often near, but steps of
        // 76 tiles pass many buckets of one tile
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
        r.e = s.cursor;
    }
    const int local = t - s.start[r.e], fill = s.fill[r.e];
    r.row = s.first[r.e];
    if (MODE == kWeightGrad) {
        const int mt = ceil_div(a.M, kM);
        const int n = local / mt;
        r.m0 = (local - n * mt) * kM;
        r.n0 = n * kN;
        r.n = min(kN, a.N - r.n0);
        r.from = 0;
        r.blocks = ceil_div(fill, kK);
        r.last = fill - (r.blocks - 1) * kK;
    } else {
        const int parts = ceil_div(fill, kN), steps = ceil_div(fill, kStep);
        const int m = local / parts, i = local - m * parts;
        const int each = steps / parts, longer = steps - each * parts;
        const int from = (i * each + min(i, longer)) * kStep;
        r.m0 = m * kM;
        r.n0 = r.row + from;
        r.n = min((each + (i < longer)) * kStep, fill - from);
        r.from = 0;
        r.blocks = ceil_div(a.K, kK);
        r.last = a.K - (r.blocks - 1) * kK;
    }
    return r;
}

// Leaves one pair's part of a tile's reduction.
__device__ __forceinline__ void take_part(Tile &c, int part, int parts)
{
    const int to = c.blocks * (part + 1) / parts;
    c.from = c.blocks * part / parts;
    if (to < c.blocks) c.last = kK;
    c.blocks = to - c.from;
}

// Lists the tiles: every thread of the CTA takes part.
template <int MODE> __device__ void build_schedule(const ExpertArgs &a, Schedule &s)
{
    __shared__ int s_warp[kThreads / 32], s_most[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0, most = 0;
    for (int e0 = 0; e0 < a.E; e0 += kThreads) {
        const int e = e0 + tid;
        int tiles = 0;
        if (e < a.E) {
            int64_t f = __ldg(a.off + e), c = __ldg(a.cnt + e);
            if (f < 0 || c < 0 || f > a.rows - c) {  // f + c may not fit
                // never outside the rows: the bucket is left out and reported
                atomicOr(&g_expert_error, kErrExpertBucket);
                f = c = 0;
            }
            s.first[e] = (int)f;
            s.fill[e] = (int)c;
            most = max(most, (int)c);
            tiles = bucket_tiles<MODE>(a, (int)c);
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

// Operand maps: the M side's, and the N side's with boxes of 16, 32, .. 128 rows.
// Weights' gradient: boxes of 64 x 64, the first of b for the N side; then boxes
// of 48 to 1 rows of the M and of the N side and of 16, 8, .. 1 rows of zeros, for
// the last block of a bucket.
constexpr int kTailM = 1, kTailN = 10, kZeros = 19;
template <int MODE> struct Maps {
    CUtensorMap a, b[MODE == kWeightGrad ? 24 : 8];
    CUtensorMap out;   // stored boxes
};

// What the padding of a bucket's last block is copied from.
__device__ __align__(128) uint16_t g_zero_rows[16 * 64];

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    volatile int stop;
};

template <typename T> __device__ __forceinline__ T round_to(float f);
template <> __device__ __forceinline__ float round_to<float>(float f) { return f; }
template <> __device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float f)
{
    return __float2bfloat16_rn(f);
}

template <int MODE, typename Tout, int JOIN, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
expert_kernel(const __grid_constant__ Maps<MODE> maps, ExpertArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    using B = Boxes<MODE, Tout, JOIN>;
    uint8_t *boxes = ring + kRingBytes;
    int *lists = reinterpret_cast<int *>(boxes + kStoreWarps * kBoxArea);
    Schedule sched = {lists, lists + a.E + 1, lists + 2 * a.E + 1, 0, 0};
    __shared__ Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the CTA's place in the pair, the pair's first CTA and place in the cluster
    const uint32_t cta = cluster_rank();
    const uint32_t rank = SPLIT ? cta & 1 : cta, lead = SPLIT ? cta & ~1u : 0;
    const int part = SPLIT ? (int)(cta >> 1) : 0, split = SPLIT ? a.split : 1;
    const int pair = blockIdx.x / (2 * split), pairs = gridDim.x / (2 * split);
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh.full[i], 4);   // both operands of both CTAs
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kStoreWarps);  // the storing warps of both CTAs
        }
        mbar_init(&sh.drain, 1);
        sh.stop = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 2 * kN);
    griddep_wait();  // the plan and the operands come from earlier stream work
    griddep_launch_dependents();
    build_schedule<MODE>(a, sched);  // ends with a CTA barrier
    cluster_sync();                  // both CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // A split grid has a cluster for each tile that disjoint buckets can have;
    // what overlapping ones have beyond is left out and reported.
    if (SPLIT && tid == 0 && sched.start[a.E] > pairs) atomicOr(&g_expert_error, kErrExpertBucket);
    const int tiles = SPLIT ? min(sched.start[a.E], pairs) : sched.start[a.E];
    // Six stages of 128 + 128 rows.  Buckets of a few rows need less of a stage,
    // and more of them keep more of the weights in flight.
    const int rows_b =
        MODE == kWeightGrad ? kN / 2 : min(kN / 2, ceil_div(sched.widest, kStep) * (kStep / 2));
    const int stage_bytes = kABytes + rows_b * 128;
    const int stages = min(kMaxStages, kRingBytes / stage_bytes);
    constexpr bool kAMn = MODE != kForward, kBMn = MODE == kWeightGrad;

    // In f32 a storing thread holds up to 128 sums.  The block starts with 384 x
    // 168 = 64512 registers; 128 x 48 + 256 x 224 = 63488.
    constexpr bool kRegs = sizeof(Tout) == 4;
    if (warp < 4) {
        if (kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 0 || warp == 2) {
            const bool weights = warp == 0;  // the M side's operand, or the N side's
            if (elect_one()) {
                const uint32_t full = addr_in(sh.full, lead);
                Ring r(stages);
                int64_t j = 0;  // blocks copied
                bool ok = true;
                for (int t = pair; t < tiles && ok; t += pairs) {
                    Tile c = tile_of<MODE>(a, sched, t);
                    if (SPLIT) take_part(c, part, split);
                    const int half = ceil_div(c.n, kStep) * (kStep / 2);
                    const int m = c.m0 + rank * kLanes, n = c.n0 + rank * half;
                    const int size = half / 16 - 1;  // the box of just this many rows
                    const int chunks = ceil_div(half, 64);
                    const uint32_t bytes = weights              ? kABytes
                                           : MODE == kWeightGrad ? chunks * 8192
                                                                 : half * 128;
                    for (int b = 0; b < c.blocks; ++b, ++j) {
                        if (j >= stages && !wait(&sh.empty[r.at], r.round ^ 1, &sh.stop)) {
                            ok = false;
                            break;
                        }
                        uint8_t *sa = ring + r.at * stage_bytes, *sb = sa + kABytes;
                        const uint32_t bar = full + r.at * 8;
                        const bool tail =
                            MODE == kWeightGrad && b + 1 == c.blocks && c.last % 16;
                        arrive_expect_at(bar, tail ? bytes / kK * tail_rows(c.last) : bytes);
                        const int k = ((SPLIT ? c.from : 0) + b) * kK;
                        if (weights) {
                            if (MODE == kForward) {
                                tma_3d(sa, &maps.a, bar, k, m, c.e);
                            } else if (MODE == kRowGrad) {
                                tma_3d(sa, &maps.a, bar, m, k, c.e);
                                tma_3d(sa + 8192, &maps.a, bar, m + 64, k, c.e);
                            } else if (tail) {
                                for (int i = 0; i < 2; ++i)
                                    tma_tail(sa + i * 8192, maps.b + kTailM, maps.b + kZeros, bar,
                                             m + i * 64, c.row + k, c.last);
                            } else {
                                tma_2d(sa, &maps.a, bar, m, c.row + k);
                                tma_2d(sa + 8192, &maps.a, bar, m + 64, c.row + k);
                            }
                        } else if (tail) {
                            for (int i = 0; i < chunks; ++i)
                                tma_tail(sb + i * 8192, maps.b + kTailN, maps.b + kZeros, bar,
                                         n + i * 64, c.row + k, c.last);
                        } else if (MODE == kWeightGrad) {
                            for (int i = 0; i < chunks; ++i)
                                tma_2d(sb + i * 8192, &maps.b[0], bar, n + i * 64, c.row + k);
                        } else {
                            tma_2d(sb, &maps.b[size], bar, k, n);
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
            // One thread waits and issues: lanes of a warp could give up a wait apart.
            if (elect_one()) {
                Ring r(stages);
                int i = -1;  // accumulators begun, less one
                bool ok = true;
                // an accumulator that the storing warps have read
                auto begin = [&] {
                    ++i;
                    if (i >= 2 &&
                        !wait(&sh.acc_empty[i & 1], (uint32_t)(i / 2 - 1) & 1, &sh.stop))
                        return false;
                    tc_fence_after();
                    return true;
                };
                auto end = [&] { mma_commit(&sh.acc_full[i & 1], lead); };
                for (int t = pair; t < tiles && ok; t += pairs) {
                    Tile c = tile_of<MODE>(a, sched, t);
                    if (SPLIT) take_part(c, part, split);
                    if (!begin()) break;
                    const int cols = ceil_div(c.n, kStep) * kStep;
                    const uint32_t idesc = instr_desc(cols, kAMn, kBMn);
                    const int parts = reduction_parts<Tout, LONG>(c.blocks);
                    int p = 1, from = 0, until = c.blocks / parts;  // blocks of part 1
                    for (int b = 0; b < c.blocks; ++b) {
                        if ((sizeof(Tout) == 4 || LONG) && b == until) {
                            end();
                            ++p;
                            from = until;
                            until = (int)((int64_t)c.blocks * p / parts);
                            ok = begin();
                            if (!ok) break;
                        }
                        if (!wait(&sh.full[r.at], r.round, &sh.stop)) {
                            ok = false;
                            break;
                        }
                        uint8_t *sa = ring + r.at * stage_bytes;
                        const int len = b + 1 == c.blocks ? c.last : kK;
                        const int steps = ceil_div(len, 16);
                        tc_fence_after();
                        const uint64_t da = operand_desc(smem_u32(sa), kAMn);
                        const uint64_t db = operand_desc(smem_u32(sa + kABytes), kBMn);
                        for (int s = 0; s < steps; ++s)
                            mma_bf16(tmem + (i & 1) * kN, da + s * (kAMn ? 128 : 2),
                                     db + s * (kBMn ? 128 : 2), idesc, b > from || s > 0);
                        mma_commit(&sh.empty[r.at], lead);
                        r.next();
                    }
                    if (ok) end();
                }
                mma_commit(&sh.drain, lead);  // nothing is issued after this
            }
            __syncwarp();
        } else if (warp == 3 && MODE != kWeightGrad) {
            zero_gaps(a.out, (int64_t)a.M * (int)sizeof(Tout), a.rows, a.cnt, a.off, a.E,
                      blockIdx.x, gridDim.x);
        }
        __syncwarp();
        if (SPLIT) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        if (kRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3;
        constexpr int kBoxRows = B::kRows;
        const int odd = warp >> 2 & 1;  // this warp's blocks of 32 columns: even or odd ones
        // the box's first storing warp and this one's place in it
        const int member = q % JOIN;
        Tout *box = reinterpret_cast<Tout *>(boxes + (warp - 4 - member) * kBoxArea);
        const bool issuer = member == 0 && lane == 0;
        auto meet = [&] {
            if (JOIN == 1)
                __syncwarp();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + odd), "n"(32 * JOIN) : "memory");
        };
        // whether all of them go on: one that gave up must not leave the others
        // at their next meeting.  Lanes may leave a wait apart, and meet as whole warps.
        auto agree = [&](bool ok) {
            if (JOIN == 1) return (bool)__all_sync(0xffffffffu, ok);
            uint32_t all;
            __syncwarp();
            asm volatile("{\n\t.reg .pred p, q;\n\t"
                         "setp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, %2, %3, p;\n\t"
                         "selp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"((uint32_t)ok), "r"(1 + odd), "n"(32 * JOIN)
                         : "memory");
            return all != 0;
        };
        int i = 0, turn = 0;
        for (int t = pair; SPLIT || t < tiles; t += pairs) {
            Tile c = SPLIT && t >= tiles ? Tile{} : tile_of<MODE>(a, sched, t);
            const int m = c.m0 + rank * kLanes + q * 32;
            const int last = (ceil_div(c.n, 32) - 1 - odd) / 2;  // last block, if any
            // columns n .. n + 32 of the output, from registers
            auto store = [&](int n, const uint32_t(&r)[32]) {
                const int m_box = m - member * 32;  // the same for all warps of a box
                if (m_box >= a.M) return;
#pragma unroll
                for (int h = 0; h < 32; h += kBoxRows) {
                    if (n + h >= c.n) break;
                    if (MODE == kWeightGrad || n + h + kBoxRows <= c.n) {
                        Tout *b = box + turn * (kBoxRows * B::kWidth);
                        if (++turn == B::kTurns) turn = 0;
                        if (issuer) bulk_wait_read<B::kTurns - 1>();
                        meet();
#pragma unroll
                        for (int x = 0; x < kBoxRows; ++x)
                            b[x * B::kWidth + member * 32 + lane] =
                                round_to<Tout>(__uint_as_float(r[h + x]));
                        fence_proxy_async_smem();
                        meet();
                        if (issuer) {
                            tma_store(&maps.out, b, m_box, c.n0 + n + h, c.e, MODE == kWeightGrad);
                            bulk_commit();
                        }
                    } else if (m + lane < a.M) {
                        // the bucket ends inside the box: the rows after it are not ours
                        Tout *out = reinterpret_cast<Tout *>(a.out) +
                                    (int64_t)(c.n0 + n + h) * a.M + m + lane;
#pragma unroll
                        for (int x = 0; x < kBoxRows; ++x, out += a.M)
                            if (n + h + x < c.n)
                                *out = round_to<Tout>(__uint_as_float(r[h + x]));
                    }
                }
            };
            if constexpr (SPLIT) {
                // One tile a cluster, of at most 64 columns: a block a warp.  Each
                // pair sums its part of the reduction; the first one adds the
                // others' in their order.
                take_part(c, part, split);
                const int n = odd * 32;
                uint32_t sum[32] = {};  // f32
                bool ok = true;
                for (int p = c.n ? reduction_parts<Tout, LONG>(c.blocks) : 0; p > 0 && ok; --p, ++i) {
                    const int buf = i & 1;
                    ok = wait_warp(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t v[32];
                    tmem_load(tmem + ((uint32_t)(q * 32) << 16) + buf * kN + n, v);
                    tmem_wait(v);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        sum[x] = __float_as_uint(__uint_as_float(sum[x]) + __uint_as_float(v[x]));
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(addr_in(&sh.acc_empty[buf], lead));
                }
                // the ring of every pair is idle now and takes the others' sums
                cluster_sync();
                const uint32_t place = (uint32_t)(n * kLanes + q * 32 + lane) * 4;
                if (part > 0 && ok && n < c.n) {
                    const uint32_t to = addr_in(ring, rank) + (part - 1) * kSplitBytes + place;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + x * kLanes * 4),
                                     "r"(sum[x])
                                     : "memory");
                }
                cluster_sync();
                if (part == 0 && ok && n < c.n) {
                    for (int o = 0; o + 1 < split; ++o) {
                        const uint8_t *from = ring + o * kSplitBytes + place;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            sum[x] = __float_as_uint(
                                __uint_as_float(sum[x]) +
                                *reinterpret_cast<const float *>(from + x * kLanes * 4));
                    }
                    store(n, sum);
                }
                break;
            }
            // this warp's blocks of accumulator i, each read while the one
            // before is stored; then the next products may have it
            auto store_all = [&] {
                const int buf = i & 1;
                if (!agree(wait(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop)))
                    return false;
                tc_fence_after();
                ++i;
                const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kN;
                uint32_t v[2][32];
                if (c.n > odd * 32) {
                    tmem_load(acc + odd * 32, v[0]);
                } else {
                    tc_fence_before();
                    if (lane == 0) arrive_at(addr_in(&sh.acc_empty[buf], lead));
                }
#pragma unroll
                for (int k = 0; k < kN / 64; ++k) {
                    const int n = k * 64 + odd * 32;
                    if (n >= c.n) break;
                    tmem_wait(v[k & 1]);
                    if (k < last) {
                        tmem_load(acc + n + 64, v[(k + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();  // every lane's columns are in registers
                        if (lane == 0) arrive_at(addr_in(&sh.acc_empty[buf], lead));
                    }
                    if (MODE == kWeightGrad && c.blocks == 0) {
                        // an expert without rows: no product was issued
#pragma unroll
                        for (int x = 0; x < 32; ++x) v[k & 1][x] = 0;
                    }
                    store(n, v[k & 1]);
                }
                return true;
            };
            const int parts = reduction_parts<Tout, LONG>(c.blocks);
            if (sizeof(Tout) == 4 && parts > 1) {
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
                    const uint32_t acc =
                        tmem + ((uint32_t)(q * 32) << 16) + buf * kN + odd * 32;
#pragma unroll
                    for (int k = 0; k < kN / 64; ++k) {
                        if (k * 64 + odd * 32 >= c.n) break;
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
                            tmem_load(acc + k * 64 + h, v);
                            tmem_wait(v);
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                sum[k][h + x] = __float_as_uint(__uint_as_float(sum[k][h + x]) +
                                                                __uint_as_float(v[x]));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(addr_in(&sh.acc_empty[buf], lead));
                }
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < kN / 64; ++k) store(k * 64 + odd * 32, sum[k]);
            } else if (LONG && parts > 1) {
                float sum[kN / 64][32];
                bool ok = true;
                for (int p = 0; p < parts; ++p, ++i) {
                    const int buf = i & 1;
                    ok = agree(wait(&sh.acc_full[buf], (uint32_t)(i / 2) & 1, &sh.stop));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc =
                        tmem + ((uint32_t)(q * 32) << 16) + buf * kN + odd * 32;
#pragma unroll 1
                    for (int k = 0; k < kN / 64 && k * 64 + odd * 32 < c.n; ++k) {
                        uint32_t v[32];
                        tmem_load(acc + k * 64, v);
                        tmem_wait(v);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            sum[k][x] = p ? sum[k][x] + __uint_as_float(v[x])
                                          : __uint_as_float(v[x]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(addr_in(&sh.acc_empty[buf], lead));
                }
                if (!ok) break;
#pragma unroll 1
                for (int k = 0; k < kN / 64 && k * 64 + odd * 32 < c.n; ++k) {
                    uint32_t v[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(sum[k][x]);
                    store(k * 64 + odd * 32, v);
                }
            } else if (!store_all()) {
                break;
            }
            __syncwarp();
        }
        if (issuer) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) (void)wait_slow(&sh.drain, 0, nullptr);  // the last matrix instruction
    __syncwarp();
    cluster_sync();  // no arrival or product of the other CTA is under way
    if (tid == 0 && sh.stop) atomicOr(&g_expert_error, kErrExpertTimeout);
    if (warp == 1) tmem_free(tmem, 2 * kN);
}

// --- host ----------------------------------------------------------------------

// A map over [depth, rows, width] (2-D when depth is 0).
cudaError_t encode(CUtensorMap *map, const void *base, bool f32, int64_t width, int64_t rows,
                   int64_t depth, int box_width, int box_rows, bool swizzle)
{
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const int size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)width * size, (cuuint64_t)width * rows * size};
    const cuuint32_t box[3] = {(cuuint32_t)box_width, (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r =
        fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
           depth ? 3 : 2, const_cast<void *>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// An operand: bf16 in boxes of 64 x box_rows with the 128-byte swizzle; what
// lies outside reads as zero.
cudaError_t make_map(CUtensorMap *map, const void *base, int64_t width, int64_t rows,
                     int64_t depth, int box_rows)
{
    return encode(map, base, false, width, rows, depth, 64, box_rows, true);
}

// The maps of tma_tail over rows.
cudaError_t make_tail_maps(CUtensorMap *map, const void *base, int64_t width, int64_t rows)
{
    cudaError_t e = cudaSuccess;
    for (int s = 4; s >= 0; s -= 2)
        for (int digit = 3; digit && e == cudaSuccess; --digit)
            e = make_map(map++, base, width, rows, 0, digit << s);
    return e;
}

// g_zero_rows on the current device.
cudaError_t zero_rows(const void **p)
{
    static void *cached[kMaxCachedDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    void *at = dev >= 0 && dev < kMaxCachedDevices ? cached[dev] : nullptr;
    if (!at) {
        e = cudaGetSymbolAddress(&at, g_zero_rows);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxCachedDevices) cached[dev] = at;
    }
    *p = at;
    return cudaSuccess;
}

// Launches `clusters` clusters of as many pairs as share a tile.
template <int MODE, typename Tout, int JOIN, bool SPLIT = false, bool LONG = false>
int launch_expert(const Maps<MODE> &maps, const ExpertArgs &a, int clusters, cudaStream_t stream)
{
    static KernelCache kc;
    auto kernel = expert_kernel<MODE, Tout, JOIN, SPLIT, LONG>;
    const size_t smem = 1024 + kRingBytes + kStoreWarps * kBoxArea +
                        (3 * (size_t)a.E + 1) * sizeof(int);
    cudaError_t e = prepare_kernel(kernel, smem, kThreads, kc, nullptr);
    if (e == cudaSuccess) {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = MOE_USE_PDL;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2 * a.split;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * a.split * clusters);
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

// ra: the rows that the reduction or the columns come from; rb: the other
// rows (weights' gradient) or the weights.
template <int MODE>
int run_expert(const void *rows_a, const void *other, int64_t rows, int64_t N, int64_t D, int E,
               const int32_t *cnt, const int64_t *off, void *out, int out_dtype,
               cudaStream_t stream)
{
    if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_EINVAL;
    if (rows < 0 || rows >= ((int64_t)1 << 31) || E < 1 || E > 1024) return MOE_EINVAL;
    if (N < 1 || D < 1 || N >= (1 << 24) || D >= (1 << 24)) return MOE_EINVAL;
    if (MODE != kWeightGrad && rows == 0) return MOE_OK;  // no rows, no output
    if (!cnt || !off || !out || (rows > 0 && (!rows_a || !other))) return MOE_EINVAL;
    const int64_t M = MODE == kForward ? N : D;
    const int64_t mt = (M + kM - 1) / kM;
    const int64_t most = MODE == kWeightGrad ? mt * ((N + kN - 1) / kN) * E
                                             : mt * (rows / kN + (rows < E ? rows : E));
    if (most >= ((int64_t)1 << 30)) return MOE_EINVAL;
    if (N % 8 || D % 8 || !aligned16(rows_a) || !aligned16(other) || !aligned16(out))
        return MOE_EALIGN;
    ExpertArgs a = {};
    a.cnt = cnt;
    a.off = off;
    a.rows = rows;
    a.E = E;
    a.split = 1;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)(MODE == kForward ? D : N);
    a.out = static_cast<uint8_t *>(out);
    Maps<MODE> maps = {};
    cudaError_t e = cudaSuccess;
    if constexpr (MODE == kWeightGrad) {
        // without rows there is nothing to copy, and no address to describe
        if (rows > 0) {
            const void *zeros = nullptr;
            e = zero_rows(&zeros);
            if (e == cudaSuccess) e = make_map(&maps.a, other, D, rows, 0, 64);
            if (e == cudaSuccess) e = make_map(&maps.b[0], rows_a, N, rows, 0, 64);
            if (e == cudaSuccess) e = make_tail_maps(&maps.b[kTailM], other, D, rows);
            if (e == cudaSuccess) e = make_tail_maps(&maps.b[kTailN], rows_a, N, rows);
            for (int i = 0; i < 5 && e == cudaSuccess; ++i)
                e = make_map(&maps.b[kZeros + i], zeros, 64, 16, 0, 16 >> i);
        }
    } else {
        e = make_map(&maps.a, other, D, N, E, MODE == kForward ? kLanes : 64);
        for (int i = 0; i < 8 && e == cudaSuccess; ++i)
            e = make_map(&maps.b[i], rows_a, a.K, rows, 0, 16 * (i + 1));
    }
    const bool f32 = out_dtype == MOE_F32;
    // a bucket may have all rows
    const bool longer = !f32 && (MODE == kWeightGrad ? rows : a.K) > kLongest;
    const bool join = MODE == kWeightGrad && !f32 && D % 16 && E * N * D * 2 > (320 << 20);
    const int box_rows = f32 ? Boxes<MODE, float, 1>::kRows : Boxes<MODE, __nv_bfloat16, 1>::kRows;
    const int box = join ? 128 : 32;
    if (e == cudaSuccess)
        e = MODE == kWeightGrad ? encode(&maps.out, out, f32, D, N, E, box, box_rows, false)
                                : encode(&maps.out, out, f32, M, rows, 0, box, box_rows, false);
    if (e != cudaSuccess) {
        set_cuda_error(e);
        return MOE_ECUDA;
    }
    if constexpr (MODE != kWeightGrad) {
        // A few rows of a few small experts fill a fraction of the pairs, each
        // streaming its tile's weights at what its own copies in flight allow.
        // The pairs of a cluster then share a tile's reduction: 15 clusters of four
        // pairs run at once, or 36 of two.  One row in each of 6 buckets, 472 x
        // 4000: 17.7 -> 10.5 us (four pairs); two in each of 8, 1024 x 4096: 18.2
        // -> 13.7 us (two); with 16 and 8 blocks of reduction nothing is lost (1312
        // long: 9.3 -> 8.9 us).
        const int blocks = ceil_div(a.K, kK);
        if (rows <= kSplitRows && most <= 36 && blocks >= 8 && !longer) {
            a.split = most <= 15 && blocks >= 16 ? 4 : 2;
            return f32 ? launch_expert<MODE, float, 1, true>(maps, a, (int)most, stream)
                       : launch_expert<MODE, __nv_bfloat16, 1, true>(maps, a, (int)most, stream);
        }
    }
    const int pairs = sm_count() / 2;
    const int clusters = (int)(most < pairs ? most : pairs);
    if (f32) return launch_expert<MODE, float, 1>(maps, a, clusters, stream);
    auto launch = longer ? launch_expert<MODE, __nv_bfloat16, 1, false, true>
                         : launch_expert<MODE, __nv_bfloat16, 1>;
    if constexpr (MODE == kWeightGrad)
        if (join)
            launch = longer ? launch_expert<MODE, __nv_bfloat16, 4, false, true>
                            : launch_expert<MODE, __nv_bfloat16, 4>;
    return launch(maps, a, clusters, stream);
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT int moe_expert_gemm(const void *x, int64_t rows, const void *w, int64_t N, int64_t D,
                               int E, const int32_t *cnt, const int64_t *off, void *y,
                               int y_dtype, moe_stream_t stream)
{
    MOE_TRACE("moe_expert_gemm");
    return run_expert<kForward>(x, w, rows, N, D, E, cnt, off, y, y_dtype, (cudaStream_t)stream);
}

MOE_EXPORT int moe_expert_gemm_dgrad(const void *dy, int64_t rows, const void *w, int64_t N,
                                     int64_t D, int E, const int32_t *cnt, const int64_t *off,
                                     void *dx, int dx_dtype, moe_stream_t stream)
{
    MOE_TRACE("moe_expert_gemm_dgrad");
    return run_expert<kRowGrad>(dy, w, rows, N, D, E, cnt, off, dx, dx_dtype,
                                (cudaStream_t)stream);
}

MOE_EXPORT int moe_expert_gemm_wgrad(const void *dy, const void *x, int64_t rows, int64_t N,
                                     int64_t D, int E, const int32_t *cnt, const int64_t *off,
                                     void *dw, int dw_dtype, moe_stream_t stream)
{
    MOE_TRACE("moe_expert_gemm_wgrad");
    return run_expert<kWeightGrad>(dy, x, rows, N, D, E, cnt, off, dw, dw_dtype,
                                   (cudaStream_t)stream);
}

namespace moe {
// Reads and clears this file's device error bits.
cudaError_t read_expert_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_expert_error, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_expert_error, &zero, sizeof(uint32_t));
    return e;
}
} // namespace moe
