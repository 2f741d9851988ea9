// A whole routed layer for a few tokens, on bf16 weights in two launches.
//
//   out[s] = sum_k topk_w[s,k] * w_down[e] h,   e = topk_idx[s,k]
//   h      = silu(w_gate[e] x[s]) * (w_up[e] x[s])
// with w_up [E, 2 F, H] (gates before ups) and w_down [E, H, F]; MXFP4 weights are in
// csrc/expert_layer_mxfp4.cu.  Every sum is f32; out is rounded once.
//
// The first launch writes h of every entry (s, k), the second y = w_down h, and
// the CTA that brings the last expert's share of 32 columns sums them over k.
// Both list the experts that have tokens from topk_idx, cut their weights into tiles
// of 32 rows and hand each CTA a contiguous run of them.
//
// A tile's weights are read once, straight into registers, and bound the call: one
// token of 8 experts reads 604 MB of weights, its other data are 100 KB.  The
// eight warps of a CTA share the reduction, each 1/8 of it over all 32 rows, and
// add their sums in shared memory, in order.  A lane's next loads are issued before it
// uses the last ones, across tiles, so that the reads do not stop while the warps
// meet.  The products are those of the warp-wide matrix instruction (mma.sync,
// 16 x 8 x 16): with at most a few tokens an expert it is far from bounding, and
// takes weights from registers, where the loads put them.
//
// Lane (g, t) holds 8 elements of rows g and g + 8; the eight columns are tokens.  x
// goes in as it is.  h has more bits than bf16: it goes in as two bf16 parts (16
// bits; three parts for f32 outputs), each a column, whose sums are added.

#include "few.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;            // weight rows of a tile: two of the instruction's 16
constexpr int kDepth = 2;            // chunks of 64 bytes of each row in flight
constexpr int kMaxRows = 8;          // tokens of an expert taken at once
constexpr int kChunk = 32;           // elements of 64 bytes of weights
constexpr int kStageBudget = 88 << 10;  // so that two CTAs fit an SM

struct LayerArgs {
    const uint8_t *x;        // bf16 [S, H]
    const int32_t *idx;      // [S, K]
    const float *topk_w;     // [S, K]
    const uint8_t *w;        // this launch's weights
    float *h;                // [S K, F]
    float *y;                // [S K, H]
    uint32_t *arrived;       // [ceil(H / 32)] experts whose share of these columns is there
    uint8_t *out;            // [S, H]
    int S, K, E, H, F;
    int rows;                // tokens of an expert taken at once
    int pitch;               // bytes of a staged row of one warp
    int out_f32;
};

// How many rows of x or h, in so many parts each, the instruction's eight columns
// hold, and the columns of one.
template <int PARTS> struct Columns {
    static constexpr int kStride = PARTS == 3 ? 4 : PARTS;
    static constexpr int kRows = 8 / kStride;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
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
template <bool UP, int PARTS>
__device__ void stage(const LayerArgs &a, const int16_t *entries, int rows, int from, int len,
                      int K, uint8_t *to)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int r = 0; r < rows; ++r) {
        const int entry = entries[r];
        uint8_t *p = to + r * PARTS * a.pitch;
        for (int k = lane * 8; k < len; k += 256) {
            float f[8];
            load8<UP>(a, entry, from + k, K, f);
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
                    if (part + 1 < PARTS) {
                        const float lo = __uint_as_float(u[i] << 16),
                                    hi = __uint_as_float(u[i] & 0xffff0000u);
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

template <bool UP, int PARTS, int NT>
__global__ void __launch_bounds__(kThreads, 2) layer_kernel(LayerArgs a)
{
    using Co = Columns<PARTS>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n = a.S * a.K;
    // shared memory: staged rows, the warps' sums (twice), the routing
    const int staged_rows = a.rows * PARTS;
    uint8_t *mine = smem + warp * staged_rows * a.pitch;
    float *sums = reinterpret_cast<float *>(smem + kWarps * staged_rows * a.pitch);
    float *weights = sums + 2 * kWarps * kMaxRows * kTile;  // of the entries
    Routing rt(weights + n, n, a.E);
    __shared__ int s_last;

    const int K = UP ? a.H : a.F;                    // reduction
    const int M = UP ? 2 * a.F : a.H;                // weight rows of an expert
    const int per_tile = UP ? kTile / 2 : kTile;     // outputs of a tile
    const int outputs = UP ? a.F : a.H;
    const int tiles = (outputs + per_tile - 1) / per_tile;
    const int row_bytes = K * 2;
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
    if (!UP) load_weights(a.topk_w, n, weights);
    route<kThreads>(a.idx, n, a.E, a.rows, rt);
    const int64_t items = (int64_t)rt.hits * tiles;
    const int begin = (int)(items * blockIdx.x / gridDim.x);
    const int end = (int)(items * (blockIdx.x + 1) / gridDim.x);

    auto advance = [&](Cursor &c) {
        if (++c.chunk < steps) return false;
        c.chunk = 0;
        const int h = c.item / tiles;
        if (++c.pass == rt.parts[h + 1] - rt.parts[h]) {
            c.pass = 0;
            ++c.item;
        }
        return true;
    };

    // --- loads ---
    uint4 w[kDepth][4];     // rows g, g + 8 of both halves of the tile
    Cursor ahead = {begin, 0, 0};
    const uint8_t *from = nullptr;
    uint32_t ok = 0;        // which of the four rows exist
    const int64_t half = (int64_t)(UP ? a.F : kTile / 2) * row_bytes;  // between the halves
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
    };
    auto load = [&](int d) {
        const int at = (c0 + ahead.chunk) * 64 + t * 16;
        const bool in = ahead.item < end && ahead.chunk < mc && at < row_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[d][i] = make_uint4(0, 0, 0, 0);
            if (in && (ok >> i & 1))
                w[d][i] = ld_stream16(from + (i & 1) * 8 * (int64_t)row_bytes + (i >> 1) * half +
                                      ahead.chunk * 64);
        }
        if (ahead.item < end && advance(ahead)) aim();
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
    int staged = -1;                  // first row of what is staged
    int first = 0, rows = 0, need = 0;  // of this visit
    int turn = 0;
    auto visit = [&] {
        if (now.item >= end) return;
        const int h = now.item / tiles;
        first = rt.first[h] + now.pass * a.rows;
        rows = min(a.rows, rt.first[h + 1] - first);
        need = (rows + Co::kRows - 1) / Co::kRows;
        if (first != staged)
            stage<UP, PARTS>(a, rt.order + first, rows, c0 * kChunk, mc * kChunk, K, mine);
        staged = first;
    };
    visit();

    auto products = [&](int d) {
        if (now.chunk >= mc) return;
        const uint8_t *b0 = mine + now.chunk * 64 + t * 16;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j >= need) break;
            // column g: part g % kStride of row g / kStride, or a column that is not used
            const int row = j * Co::kRows + g / Co::kStride, part = g % Co::kStride;
            uint4 b = make_uint4(0, 0, 0, 0);
            if (row < rows && part < PARTS)
                b = *reinterpret_cast<const uint4 *>(b0 + (row * PARTS + part) * a.pitch);
            // The instruction cuts a sum's low bits off: after 100 of them an f32
            // output is off by 1e-6.  Two at a time, added in f32, 2e-7.
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint4 u = w[d][2 * m], v = w[d][2 * m + 1];
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma(c, u.x, v.x, u.y, v.y, b.x, b.y);
                mma(c, u.z, v.z, u.w, v.w, b.z, b.w);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] += c[i];
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
                const float (&v)[4] = acc[m][j];
                const int at = m * 16 + g;
                if (PARTS == 1) {
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
        const int tile = item % tiles, o = tile * kTile + lane;
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(a.arrived + tile, 1u) == (uint32_t)rt.hits - 1;
            __threadfence();
        }
        __syncthreads();
        if (!s_last || o >= a.H) return;
        // a token a warp where that is enough
        const int each = a.S > kWarps ? kFewTokens : 1;
        for (int s0 = warp * each; s0 < a.S; s0 += kWarps * each) {
            int s[kFewTokens];
#pragma unroll
            for (int j = 0; j < kFewTokens; ++j) s[j] = min(s0 + j, a.S - 1);
            if (each == 1)
                few_combine<1>(a.y, weights, rt.place, a.K, a.H, o, s, 1, a.out, a.out_f32);
            else
                few_combine<kFewTokens>(a.y, weights, rt.place, a.K, a.H, o, s, a.S - s0, a.out,
                                        a.out_f32);
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
                advance(now);
                if (!UP && now.item != item) combine(item);
                visit();
            } else {
                ++now.chunk;
            }
        }
    }
}

// --- host ----------------------------------------------------------------------

template <bool UP, int PARTS, int NT> int launch_layer(LayerArgs a, cudaStream_t stream)
{
    static KernelCache kc;
    auto kernel = layer_kernel<UP, PARTS, NT>;
    const int K = UP ? a.H : a.F, n = a.S * a.K;
    const int chunks = (K * 2 + 63) / 64;
    const int mine = (chunks + kWarps - 1) / kWarps;  // of one warp
    // neighbouring staged rows begin in other banks
    a.pitch = mine * 64 + (mine % 2 ? 0 : 64);
    const int row = kWarps * PARTS * a.pitch;
    int rows = kStageBudget / row;
    const int most = NT * Columns<PARTS>::kRows < kMaxRows ? NT * Columns<PARTS>::kRows : kMaxRows;
    if (rows > most) rows = most;
    if (rows > a.S) rows = a.S;  // more only where a token has an expert twice
    a.rows = rows < 1 ? 1 : rows;
    const size_t smem = (size_t)a.rows * row + 2 * kWarps * kMaxRows * kTile * 4 + n * 4 +
                        Routing::bytes(n, a.E);
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

// The workspace: y, h and the counters.
struct Places {
    int64_t h, arrived, bytes;
    Places(int64_t n, int64_t H, int64_t F)
    {
        h = round_up(n * H * 4, 256);
        arrived = h + round_up(n * F * 4, 256);
        bytes = arrived + round_up((H + kTile - 1) / kTile * 4, 256);
    }
};

int layer_bf16(const LayerCall &c, cudaStream_t stream)
{
    const Places at(c.S * c.K, c.H, c.F);
    LayerArgs a = {};
    a.x = c.x;
    a.idx = c.idx;
    a.topk_w = c.topk_w;
    a.w = c.up;
    a.y = reinterpret_cast<float *>(c.workspace);
    a.h = reinterpret_cast<float *>(c.workspace + at.h);
    a.arrived = reinterpret_cast<uint32_t *>(c.workspace + at.arrived);
    a.out = c.out;
    a.S = c.S;
    a.K = c.K;
    a.E = c.E;
    a.H = c.H;
    a.F = c.F;
    a.out_f32 = c.f32;
    const int r = launch_layer<true, 1, 1>(a, stream);
    if (r != MOE_OK) return r;
    a.w = c.down;
    return c.f32 ? launch_layer<false, 3, 4>(a, stream) : launch_layer<false, 2, 2>(a, stream);
}

bool in_range(int64_t S, int64_t H, int K, int E, int64_t F)
{
    return S >= 0 && K >= 1 && K <= 32 && E >= 1 && E <= kFewExperts && H >= 1 && F >= 1 &&
           H <= kFewWidth && F <= kFewWidth && S <= kFewEntries && S * K <= kFewEntries;
}

} // namespace
} // namespace moe

using namespace moe;

MOE_EXPORT size_t moe_expert_layer_workspace_size(int64_t S, int64_t H, int K, int E, int64_t F,
                                                  int w_dtype)
{
    if (!in_range(S, H, K, E, F)) return 0;
    if (w_dtype == MOE_MXFP4) return layer_mxfp4_workspace(S, K, E, H, F);
    return w_dtype == MOE_BF16 ? (size_t)Places(S * K, H, F).bytes : 0;
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
    const LayerCall c = {static_cast<const uint8_t *>(x),
                         topk_idx,
                         topk_w,
                         static_cast<const uint8_t *>(w_up),
                         up_scales,
                         static_cast<const uint8_t *>(w_down),
                         down_scales,
                         static_cast<uint8_t *>(out),
                         static_cast<uint8_t *>(workspace),
                         (int)S,
                         K,
                         E,
                         (int)H,
                         (int)F,
                         f32};
    return mx ? layer_mxfp4(c, (cudaStream_t)stream) : layer_bf16(c, (cudaStream_t)stream);
}
