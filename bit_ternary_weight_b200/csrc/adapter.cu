// adapter.cu -- low-rank adapters of many requests beside one shared
// projection: out[t] = y[t] + scale[a] up[a] (down[a] x[t]), a = index[t].
//
// Two launches, the second chained to the first (programmatic dependent
// launch): u[t] = scale[a] down[a] x[t] in fp32 to the workspace, then
// out = y + up u; with more than 128 tokens a third before them, which brings
// tokens of one adapter together.  Both products are bound by memory: a token brings 2 r (K + N)
// multiply-adds against 2 K + 4 N bytes, and a few tokens bring their whole
// adapters, so the products run as mma.sync m16n8k16 straight from registers
// (r columns or r terms are far too few for a tcgen05 tile) and the work is
// in keeping loads in flight:
//   - a tile is 16 tokens (the first launch takes two tiles a CTA where there
//     are enough); the tokens' distinct adapters are found with one
//     match across the warp and taken one after the other, each giving only
//     its own tokens' rows (the other rows of its products are dropped, so
//     nothing of an adapter reaches a token that does not use it);
//   - a sum does not mind the order of its terms, so the k index of an MMA is
//     permuted such that each lane's operands are contiguous: 16 bytes of x
//     and of down (8 consecutive k of a 32-k group, two MMAs), 8 bytes of up
//     (4 consecutive ranks); the same for the output columns (four n8 tiles
//     interleaved give a lane 8 consecutive columns of y and out).
// With few tokens the adapters of a tile go to different CTAs (first launch)
// or warps (second), and K is split over CTAs whose partial sums the second
// launch adds in order: the same call gives the same bits.
// u enters the second product as a sum of bf16 values, each the rest of the
// one before: two (16 bits of it) for bf16 outputs, three (24 bits) for fp32
// outputs; one alone would cost an output 2^-8 of the adapter's share.
// Measured (inputs that change from call to call): 4093 tokens of prompts, 2560
// to 6912 columns, rank 16, 136 MB: 44.7 us, 3.0 TB/s, of which the order takes 1,
// the first product 15 and the second 28; at rank 64 91 us.  32 tokens of 24
// adapters, 2560 x 2560: 10.7 us, a token at rank 64 (fp32): 7.6 us, three to four
// memory latencies in a row each.  Ranks above 64 are the ones without room: the
// second product's kernels hold 64 registers of `up` a lane and spill up to 168
// bytes at 128 registers, and take a tile at a time: 170 us at rank 72, 204 at
// 128 for the prompts; 18 and 21 us for the 32 tokens.
#include <algorithm>

#include "bl_common.cuh"

namespace bl {
namespace {

constexpr int kTile = 16;                 // tokens per tile (MMA M)
constexpr int kDownWarps = 8, kUpWarps = 8;
constexpr int kUpCols = 32;               // output columns per warp
constexpr int kChunk = 1024;              // tokens that are sorted together

struct AdapterParams {
    const void *y;
    int64_t ldy;
    const __nv_bfloat16 *x;
    int64_t ldx, T, N, K;
    const __nv_bfloat16 *down, *up;
    int n, r;
    const int32_t *index;
    const float *scale;
    void *out;
    int64_t ldo;
    float *u;                             // [splits][T][r]
    int2 *order;                          // (token, adapter) in the order of the tiles; null: as they come
    int splits;
    int down_ways;                        // CTAs that share the adapters of a tile
    int *status;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The adapter of token t, -1: none; an id that does not exist counts as none.
__device__ __forceinline__ int token_id(const AdapterParams &p, int64_t t, bool report)
{
    int id = int(ld_dep_u32(p.index + t));
    if (id >= p.n) {
        if (report)
            atomicExch(p.status, BL_ERR_SHAPE);
        id = -1;
    }
    return id < 0 ? -1 : id;
}

// The token at place `at` of the tiles' order and its adapter.
__device__ __forceinline__ int2 placed(const AdapterParams &p, int64_t at, bool report)
{
    if (!p.order)
        return make_int2(int(at), token_id(p, at, report));
    return __ldcg(p.order + at);
}

// Lanes that are the first with their adapter.
__device__ __forceinline__ unsigned first_of(int id, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, id);
    return __ballot_sync(0xffffffffu, id >= 0 && lane == __ffs(same) - 1);
}

// The order in which tokens go to tiles, for many tokens.  Where tokens of many
// adapters alternate (requests' single tokens), a tile of consecutive ones takes
// a product per adapter, up to 16; sorted by adapter within 1024 tokens it takes
// one or two.  Tokens that come in runs (prompts) stay in place.  A stable
// counting sort on 255 bins, so the order depends on the ids alone; adapters
// that share a bin (id mod 255) only share tiles, tokens without one come last.
// 4096 tokens of 16 adapters, 2560 x 2560, rank 16: 140 -> 31 us with it.
__global__ void __launch_bounds__(kChunk) adapter_order_kernel(const AdapterParams p)
{
    constexpr int kBins = 256, kWarps = kChunk / 32;
    __shared__ uint16_t count[kWarps][kBins];     // of a warp's tokens; then what precedes them in the bin
    __shared__ int base[kBins], warp_sum[kBins / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < kWarps * kBins / 8; e += kChunk)
        reinterpret_cast<uint4 *>(&count[0][0])[e] = make_uint4(0, 0, 0, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t c0 = int64_t(blockIdx.x) * kChunk, t = c0 + tid;
    const int id = t < p.T ? token_id(p, t, true) : -1, bin = id < 0 ? kBins - 1 : id % (kBins - 1);
    const unsigned peers = __match_any_sync(0xffffffffu, bin);
    const int rank = __popc(peers & ((1u << lane) - 1));
    // the products that the chunk's tiles take as they come: worth an order above
    // three for two tiles (2 adapters, alternating: 40 -> 28 us; prompts, which
    // an order would only move: 27 -> 31)
    const unsigned half = lane < kTile ? 0x0000ffffu : 0xffff0000u;
    const int products = __syncthreads_count(id >= 0 && !(peers & half & ((1u << lane) - 1)));
    const int tiles = int(min(int64_t(kChunk), p.T - c0) + kTile - 1) / kTile;
    int place = tid;
    if (2 * products > 3 * tiles) {
        if (rank == 0)
            count[warp][bin] = uint16_t(__popc(peers));
        __syncthreads();
        int sum = 0, scan = 0;                    // of bin tid
        if (tid < kBins) {
#pragma unroll 8
            for (int w = 0; w < kWarps; ++w) {
                const int c = count[w][tid];
                count[w][tid] = uint16_t(sum);
                sum += c;
            }
            scan = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, scan, o);
                scan += lane >= o ? v : 0;
            }
            if (lane == 31)
                warp_sum[warp] = scan;
        }
        __syncthreads();
        if (tid < kBins) {
            for (int w = 0; w < warp; ++w)
                scan += warp_sum[w];
            base[tid] = scan - sum;
        }
        __syncthreads();
        place = base[bin] + count[warp][bin] + rank;
    }
    // places behind the last token stay there: they are the last of the last bin
    if (t < p.T)
        __stcg(p.order + c0 + place, make_int2(int(t), id));
}

// u of MT tiles, one K split: RW warps side by side have 8 NT ranks each, and
// 8 / RW take the split's 32-k groups in turn; their sums are added through
// shared memory in a fixed order.  With many tokens a CTA takes MT = 2 tiles,
// which share what they read of an adapter: 4096 tokens, 2560 x 2560, rank 64,
// 59 us instead of 97, rank 16 27 instead of 29 (4 tiles: 33, registers spill).
template <int NT, int RW, int MT>
__global__ void __launch_bounds__(kDownWarps * 32, 2) adapter_down_kernel(const AdapterParams p)
{
    constexpr int kWays = kDownWarps / RW;                    // warps that share the k groups
    constexpr int kRows = MT * kTile;
    static_assert(kRows <= 32, "a lane per row");
    __shared__ __align__(16) float red[kWays / 2][kRows][RW * NT * 8];
    // the second launch reads y before it waits for this one, so it may begin
    // only when what came before this one is complete
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = int64_t(blockIdx.x) * kRows;
    const int valid = int(min(int64_t(kRows), p.T - t0));
    const int way = blockIdx.y, split = blockIdx.z;
    const int groups = int(p.K / 32), kw = warp / RW, r0 = warp % RW * NT * 8;
    const int k0 = int(int64_t(split) * groups / p.splits) + kw, k1 = int(int64_t(split + 1) * groups / p.splits);
    constexpr int kDeep = MT > 1 || NT > 2 ? 2 : 4;           // groups in flight
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // all tokens' x, before their adapters are known: the rows of other
    // adapters are dropped at the end
    int token[MT][2];                                         // -1: behind the last
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m)
        token[m / 2][m % 2] = 8 * m + g < valid ? int(t0) + 8 * m + g : -1;
    uint4 x[kDeep][MT][2];
    auto load_x = [&](int k) {
#pragma unroll
        for (int s = 0; s < kDeep; ++s) {
            const __nv_bfloat16 *at = p.x + int64_t(k + s * kWays) * 32 + 8 * c;
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) {
                const int t = token[m / 2][m % 2];
                x[s][m / 2][m % 2] = k + s * kWays < k1 && t >= 0 ? ld_dep_v4(at + t * p.ldx) : zero;
            }
        }
    };
    load_x(k0);
    const int2 mine = lane < valid ? placed(p, t0 + lane, way == 0 && split == 0) : make_int2(-1, -1);
    if (p.order) {
        // and again where other tokens than the consecutive ones are the tiles'
        bool moved = false;
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
            const int t = __shfl_sync(0xffffffffu, mine.x, 8 * m + g);
            moved |= t != token[m / 2][m % 2];
            token[m / 2][m % 2] = t;
        }
        if (__any_sync(0xffffffffu, moved))
            load_x(k0);
    }
    int held = k0;                                            // x of the groups from here on is in registers
    const int id = mine.y;
    unsigned firsts = first_of(id, lane);
    for (int ord = 0; firsts; ++ord, firsts &= firsts - 1) {
        if (ord % p.down_ways != way)
            continue;
        const int a = __shfl_sync(0xffffffffu, id, __ffs(firsts) - 1);
        const unsigned rows = __ballot_sync(0xffffffffu, id == a);
        const __nv_bfloat16 *w = p.down + (int64_t(a) * p.r + r0 + g) * p.K + 8 * c;
        float acc[MT][NT][4] = {};
        for (int k = k0; k < k1; k += kDeep * kWays) {
            uint4 b[kDeep][NT];
            if (k != held)
                load_x(held = k);
#pragma unroll
            for (int s = 0; s < kDeep; ++s) {
                const int64_t at = int64_t(k + s * kWays) * 32;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b[s][j] = k + s * kWays < k1 && r0 + j * 8 < p.r ? ld_ro_v4(w + j * 8 * p.K + at) : zero;
            }
#pragma unroll
            for (int s = 0; s < kDeep; ++s) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 xa = x[s][m][0], xb = x[s][m][1];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        mma_bf16(acc[m][j], xa.x, xb.x, xa.y, xb.y, b[s][j].x, b[s][j].y);
                        mma_bf16(acc[m][j], xa.z, xb.z, xa.w, xb.w, b[s][j].z, b[s][j].w);
                    }
                }
            }
        }
        // sums of the first and the second half of the k ways, then of all pairs
        const int pair = kw % (kWays / 2);
        for (int half = 1; half >= 0; --half) {
            if (kw / (kWays / 2) == half) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float2 &s = *reinterpret_cast<float2 *>(&red[pair][16 * m + g + 4 * e][r0 + 8 * j + 2 * c]);
                            const float2 v = make_float2(acc[m][j][e], acc[m][j][e + 1]);
                            s = half ? v : make_float2(s.x + v.x, s.y + v.y);
                        }
                    }
                }
            }
            __syncthreads();
        }
        const float scale = p.scale ? __ldcg(p.scale + a) : 1.0f;
        const int fours = p.r / 4;
        for (int e = threadIdx.x; e < kRows * fours; e += kDownWarps * 32) {
            const int at = e / fours, j = 4 * (e - at * fours);
            if (rows >> at & 1) {
                float4 s = *reinterpret_cast<const float4 *>(&red[0][at][j]);
#pragma unroll
                for (int q = 1; q < kWays / 2; ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(&red[q][at][j]);
                    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
                }
                __stcg(reinterpret_cast<float4 *>(p.u + (int64_t(split) * p.T + t0 + at) * p.r + j),
                       make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale));
            }
        }
        __syncthreads();
    }
}

// Eight consecutive elements of a row of whole 16-byte vectors.
template <bool F32>
struct Cols {
    uint4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const char *src)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            v[i] = ld_dep_v4(src + 16 * i);
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const
    {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        if constexpr (F32) {
            const uint32_t z[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = __uint_as_float(w[i]);
                f[4 + i] = __uint_as_float(z[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    // The elements as they were loaded.
    __device__ __forceinline__ void copy(char *dst) const
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            reinterpret_cast<uint4 *>(dst)[i] = v[i];
    }
    static __device__ __forceinline__ void store(char *dst, const float (&f)[8])
    {
        if constexpr (F32) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                         pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
    }
};

// a's first bf16 term, and a without it: an infinity or a NaN is its own first
// term and leaves nothing (not inf - inf), and a finite value that would round
// to infinity takes the largest finite bf16 and the rest.
__device__ __forceinline__ float first_term(float a, float &rest)
{
    constexpr float kMax = 3.38953139e38f;                    // 0x7f7f0000
    const bool finite = fabsf(a) <= 3.40282347e38f;
    const float t = __bfloat162float(__float2bfloat16_rn(finite ? fminf(fmaxf(a, -kMax), kMax) : a));
    rest = finite ? a - t : 0.0f;
    return t;
}

// The values (a, b) as sums of TERMS bf16 values, largest first.
template <int TERMS>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&w)[TERMS])
{
    float ra, rb;
    const float ta = first_term(a, ra), tb = first_term(b, rb);
    w[0] = pack_bf16(ta, tb);
#pragma unroll
    for (int i = 1; i < TERMS; ++i) {
        w[i] = pack_bf16(ra, rb);
        ra -= __uint_as_float(w[i] << 16);
        rb -= __uint_as_float(w[i] & 0xffff0000u);
    }
}

// out = y + up u for runs of TILES tiles and the columns of a CTA.  A warp has
// 32 columns; WAYS = 1: the warps of a CTA lie side by side and take a run's
// tiles one after the other, every tile's y in flight from the start; WAYS = 8:
// they share 32 columns and the adapters of one tile.  y and the adapters are
// asked for while the first launch still runs.  u, the K splits' parts added
// in order, is split into its bf16 terms once per CTA, and the operand of the
// last adapter stays from tile to tile (prompts).  For bf16 rows of whole
// 16-byte vectors the accumulators start at y; fp32 rows (a tensor core's sums
// would lose up to 2^-23 of y each) and rows that are not whole vectors add y at
// the end.  Which of the two goes by the row layout and the type, whichever tokens
// share the tile, so that a token gets the same bits beside any others where the
// K splits are the same.  Rows that are not whole vectors (VEC = false) go through
// shared memory, so that a warp reads and writes 32 columns of a row at once:
// 4096 tokens, 704 x 1001, rank 16, 26 us instead of 35 with a lane's eight
// columns one by one.
template <int KB, bool F32, int WAYS, int TILES, bool VEC>
__global__ void __launch_bounds__(kUpWarps * 32, 2) adapter_up_kernel(const AdapterParams p)
{
    static_assert(VEC || TILES == 1, "rows through shared memory: a tile at a time");
    constexpr int kTokens = TILES * kTile;
    constexpr int kTerms = F32 ? 3 : 2;
    constexpr int kPitch = 8 * KB + 4;                        // words (two ranks) per token
    __shared__ uint32_t u_s[kTerms][kTokens][kPitch];
    __shared__ int id_s[kTokens], token_s[kTokens];
    __shared__ float2 sums[VEC ? 1 : kUpWarps][kTile][VEC ? 1 : kUpCols / 2 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int way = WAYS == 1 ? 0 : warp;
    const int64_t n0 = (int64_t(blockIdx.x) * (kUpWarps / WAYS) + (WAYS == 1 ? warp : 0)) * kUpCols;
    const int64_t nc = n0 + 8 * c;                            // this lane's output columns
    const bool cols = n0 < p.N, own = nc < p.N;
    constexpr int kElem = F32 ? 4 : 2;
    const char *const yp = static_cast<const char *>(p.y);
    char *const op = static_cast<char *>(p.out);
    bool waited = false;
    uint2 b[KB][4];
    int b_of = -1;                                            // the adapter that b holds
    auto load_b = [&](int a) {
        if (a == b_of)
            return;
        b_of = a;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                // column g of tile x: 8 (g / 2) + 2 x + g % 2; this lane's four ranks
                const int64_t n = n0 + 8 * (g >> 1) + 2 * x + (g & 1);
                const int k = 16 * kb + 4 * c;
                b[kb][x] = make_uint2(0, 0);
                if (k < p.r && n < p.N)
                    b[kb][x] = __ldg(reinterpret_cast<const uint2 *>(p.up + (int64_t(a) * p.N + n) * p.r + k));
            }
        }
    };
    for (int64_t run = blockIdx.y; run * kTokens < p.T; run += gridDim.y) {
        const int64_t t0 = run * kTokens;
        const int tokens = int(min(int64_t(kTokens), p.T - t0));
        __syncthreads();                                      // the last run's u has been used
        Cols<F32> y[TILES][2];
        if constexpr (VEC) {
            const char *src = yp + ((t0 + g) * p.ldy + nc) * kElem;
            const int64_t step = 8 * p.ldy * kElem;
#pragma unroll
            for (int i = 0; i < 2 * TILES; ++i, src += step)
                if (8 * i + g < tokens && own)
                    y[i / 2][i % 2].load(src);
        }
        bool moved = false;
        if (threadIdx.x < kTokens) {
            const int2 at = int(threadIdx.x) < tokens ? placed(p, t0 + threadIdx.x, false) : make_int2(0, -1);
            token_s[threadIdx.x] = at.x;
            id_s[threadIdx.x] = at.y;
            moved = int(threadIdx.x) < tokens && at.x != t0 + threadIdx.x;
        }
        moved = __syncthreads_or(moved);
        if constexpr (VEC) {
            // again where other tokens than the consecutive ones are the run's
            if (moved) {
#pragma unroll
                for (int i = 0; i < 2 * TILES; ++i)
                    if (8 * i + g < tokens && own)
                        y[i / 2][i % 2].load(yp + (token_s[8 * i + g] * p.ldy + nc) * kElem);
            }
        }
        uint32_t w[kTile];                                    // column n0 + lane of the rows (VEC = false)
        if constexpr (!VEC) {
#pragma unroll
            for (int r = 0; r < kTile; ++r) {
                const char *src = yp + (token_s[r] * p.ldy + n0 + lane) * kElem;
                w[r] = r >= tokens || n0 + lane >= p.N ? 0u : F32 ? ld_dep_u32(src) : ld_dep_u16(src) << 16;
            }
        }
        if (WAYS == 1 && cols && id_s[0] >= 0)
            load_b(id_s[0]);
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            waited = true;
        }
        for (int e = threadIdx.x; e < tokens * 4 * KB; e += kUpWarps * 32) {
            const int row = e / (4 * KB), k = 4 * (e % (4 * KB));
            float4 s = {};                                    // ranks behind r are zeros
            if (k < p.r && id_s[row] >= 0) {
                const float *u = p.u + (t0 + row) * p.r + k;
#pragma unroll 8
                for (int z = 0; z < p.splits; ++z) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(u + int64_t(z) * p.T * p.r));
                    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
                }
            }
            uint32_t lo[kTerms], hi[kTerms];
            split_bf16(s.x, s.y, lo);
            split_bf16(s.z, s.w, hi);
#pragma unroll
            for (int q = 0; q < kTerms; ++q)
                *reinterpret_cast<uint2 *>(&u_s[q][row][k / 2]) = make_uint2(lo[q], hi[q]);
        }
        __syncthreads();
        if (!cols)
            continue;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            if (16 * i >= tokens)
                break;
            // acc += up u of adapter a for all 16 tokens (rows of other
            // adapters are dropped by the caller)
            auto product = [&](int a, float (&acc)[4][4]) {
                load_b(a);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    if (16 * kb >= p.r)
                        break;
#pragma unroll
                    for (int q = kTerms - 1; q >= 0; --q) {
                        const uint2 ua = *reinterpret_cast<const uint2 *>(&u_s[q][16 * i + g][8 * kb + 2 * c]);
                        const uint2 ub = *reinterpret_cast<const uint2 *>(&u_s[q][16 * i + g + 8][8 * kb + 2 * c]);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_bf16(acc[x], ua.x, ub.x, ua.y, ub.y, b[kb][x].x, b[kb][x].y);
                    }
                }
            };
            auto dst = [&](int h) { return op + (token_s[16 * i + 8 * h + g] * p.ldo + nc) * kElem; };
            const int id = lane < kTile ? id_s[16 * i + lane] : -1;
            const int valid = min(16, tokens - 16 * i), one = __shfl_sync(0xffffffffu, id, 0);
            if constexpr (VEC && !F32 && WAYS == 1) {
                // one adapter for all (most tiles of a prompt): what finish() does,
                // without its loop and masks (48.7 us of prompts without this)
                if (one >= 0 && __all_sync(0xffffffffu, id == one || lane >= valid)) {
                    float acc[4][4], f[8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        y[i][h].floats(f);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[e / 2][2 * h + e % 2] = f[e];
                    }
                    product(one, acc);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = acc[e / 2][2 * h + e % 2];
                        if (g + 8 * h < valid && own)
                            Cols<F32>::store(dst(h), f);
                    }
                    continue;
                }
            }
            // out = y + the product with adapter a for some of the tile's rows
            auto finish = [&](unsigned rows, int a) {
                float acc[4][4] = {};
                if constexpr (VEC) {
                    float f[2][8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        y[i][h].floats(f[h]);
                        if constexpr (!F32) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                acc[e / 2][2 * h + e % 2] = f[h][e];
                        }
                    }
                    product(a, acc);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if ((rows >> (g + 8 * h) & 1) && own) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                f[h][e] = acc[e / 2][2 * h + e % 2] + (F32 ? f[h][e] : 0.0f);
                            Cols<F32>::store(dst(h), f[h]);
                        }
                    }
                } else {
                    const int64_t n = n0 + lane;
                    rows = n < p.N ? rows : 0;
                    product(a, acc);
                    __syncwarp();                             // the last sums have been read
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            sums[warp][g + 8 * h][4 * c + x] = make_float2(acc[x][2 * h], acc[x][2 * h + 1]);
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < kTile; ++r)
                        if (rows >> r & 1)
                            store_y(op + token_s[r] * p.ldo * kElem, F32 ? BL_F32 : BL_BF16, n,
                                    __uint_as_float(w[r]) + reinterpret_cast<const float *>(sums[warp][r])[lane]);
                }
            };
            // out = y, bit for bit (a sum with zero would lose the sign of -0)
            auto keep = [&](unsigned rows) {
                if constexpr (VEC) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if ((rows >> (g + 8 * h) & 1) && own)
                            y[i][h].copy(dst(h));
                } else {
                    const int64_t n = n0 + lane;
                    rows = n < p.N ? rows : 0;
#pragma unroll
                    for (int r = 0; r < kTile; ++r) {
                        if (rows >> r & 1) {
                            char *at = op + (token_s[r] * p.ldo + n) * kElem;
                            if constexpr (F32)
                                *reinterpret_cast<uint32_t *>(at) = w[r];
                            else
                                *reinterpret_cast<uint16_t *>(at) = uint16_t(w[r] >> 16);
                        }
                    }
                }
            };
            unsigned firsts = first_of(id, lane);
            const unsigned none = __ballot_sync(0xffffffffu, lane < valid && id < 0);
            if (way == 0 && none)
                keep(none);
            for (int ord = 0; firsts; ++ord, firsts &= firsts - 1) {
                if (WAYS > 1 && ord % WAYS != way)
                    continue;
                const int a = __shfl_sync(0xffffffffu, id, __ffs(firsts) - 1);
                finish(__ballot_sync(0xffffffffu, id == a), a);
            }
        }
    }
}

// Tiles of a run: as many as leave the adapter's operand (8 KB registers) and
// the tiles' y in registers up to KB = 4; at KB = 8 one tile already spills.
constexpr int run_tiles(int kb, bool f32) { return kb > 4 ? 1 : kb > 2 ? (f32 ? 1 : 2) : f32 ? 2 : 4; }

// With fewer tokens, the adapters of a tile have warps and CTAs of their own.
constexpr int64_t kOrderTokens = 128;

// K splits of the first launch at most: eight CTAs of a tile, or two of two
// tiles, per SM (T is all the workspace's size may depend on).
int max_splits(int64_t T, int sms)
{
    const int64_t tiles = (T + kTile - 1) / kTile;
    return int(std::clamp<int64_t>(8 * sms / tiles, 1, 32));
}

// One tile a CTA or two.
auto down_kernel(int r, bool two) -> void (*)(AdapterParams)
{
    if (two)
        return r <= 8    ? adapter_down_kernel<1, 1, 2>
               : r <= 16 ? adapter_down_kernel<2, 1, 2>
               : r <= 32 ? adapter_down_kernel<4, 1, 2>
               : r <= 64 ? adapter_down_kernel<4, 2, 2>
                         : adapter_down_kernel<4, 4, 2>;
    return r <= 8    ? adapter_down_kernel<1, 1, 1>
           : r <= 16 ? adapter_down_kernel<2, 1, 1>
           : r <= 32 ? adapter_down_kernel<4, 1, 1>
           : r <= 64 ? adapter_down_kernel<4, 2, 1>
                     : adapter_down_kernel<4, 4, 1>;
}

cudaError_t launch(void (*kernel)(AdapterParams), dim3 grid, int threads, cudaStream_t s, const AdapterParams &p)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;       // each kernel waits itself for what came before it
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

enum class Up { kFew, kTile, kRun };      // eight warps a tile; a tile, a run of tiles a warp

template <int KB, bool F32>
auto up_kernel(Up kind, bool vec) -> void (*)(AdapterParams)
{
    if (kind == Up::kFew)
        return vec ? adapter_up_kernel<KB, F32, 8, 1, true> : adapter_up_kernel<KB, F32, 8, 1, false>;
    return !vec                 ? adapter_up_kernel<KB, F32, 1, 1, false>
           : kind == Up::kTile ? adapter_up_kernel<KB, F32, 1, 1, true>
                               : adapter_up_kernel<KB, F32, 1, run_tiles(KB, F32), true>;
}

template <bool F32>
auto up_kernel(int r, Up kind, bool vec) -> void (*)(AdapterParams)
{
    return r <= 16   ? up_kernel<1, F32>(kind, vec)
           : r <= 32 ? up_kernel<2, F32>(kind, vec)
           : r <= 64 ? up_kernel<4, F32>(kind, vec)
                     : up_kernel<8, F32>(kind, vec);
}

}  // namespace

size_t adapter_workspace_bytes(int64_t T, int r)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return 0;
    // A bound of max_splits(t) * t for every t up to T, since a workspace also
    // serves fewer tokens, which may be split further: tiles times splits stay
    // at 8 per SM or below unless every tile has one split.
    const int64_t rows = std::max(T, std::min(32 * T, int64_t(8) * di->sm_count * kTile));
    return size_t(rows) * size_t(r) * sizeof(float) + (T > kOrderTokens ? size_t(T) * sizeof(int2) : 0);
}

int launch_adapter_add(const AdapterArgs &a, cudaStream_t s)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return BL_ERR_CUDA;
    const int64_t tiles = (a.T + kTile - 1) / kTile;
    const int esz = a.yt == BL_BF16 ? 2 : 4;
    auto aligned = [&](const void *q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * esz % 16 == 0; };
    AdapterParams p{};
    p.y = a.y;
    p.ldy = a.ldy;
    p.x = static_cast<const __nv_bfloat16 *>(a.x);
    p.ldx = a.ldx;
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.down = static_cast<const __nv_bfloat16 *>(a.down);
    p.up = static_cast<const __nv_bfloat16 *>(a.up);
    p.n = a.n;
    p.r = a.r;
    p.index = a.index;
    p.scale = a.scale;
    p.out = a.out;
    p.ldo = a.ldo;
    p.u = static_cast<float *>(a.ws);
    // two tiles a CTA where those and the K splits (of a group a warp or more) fill the GPU
    const int64_t pairs = (tiles + 1) / 2, k_splits = a.K / 32 / kDownWarps;
    const bool two = pairs * std::min<int64_t>(k_splits, max_splits(a.T, di->sm_count)) >= di->sm_count;
    p.splits = int(std::clamp<int64_t>(two ? 2 * di->sm_count / pairs : 6 * di->sm_count / tiles, 1,
                                       std::clamp<int64_t>(k_splits, 1, max_splits(a.T, di->sm_count))));
    p.status = di->status;
    const bool ordered = a.T > kOrderTokens && a.n > 1;
    // a tile's adapters go to CTAs of their own while tiles alone do not fill the GPU
    p.down_ways = int(std::clamp<int64_t>(di->sm_count / tiles, 1, std::min<int64_t>({ordered ? 2 : kTile, a.n, a.T})));
    auto down = down_kernel(a.r, two);
    int st = BL_OK;
    if (ordered) {
        // behind u, whose size is a multiple of 16 bytes
        p.order = reinterpret_cast<int2 *>(p.u + size_t(max_splits(a.T, di->sm_count)) * a.T * a.r);
        st = cuda_status(launch(adapter_order_kernel, dim3(unsigned((a.T + kChunk - 1) / kChunk)), kChunk, s, p));
        if (st)
            return st;
    }
    const dim3 dgrid(unsigned(two ? pairs : tiles), unsigned(p.down_ways), unsigned(p.splits));
    st = cuda_status(launch(down, dgrid, kDownWarps * 32, s, p));
    if (st)
        return st;
    // rows of whole 16-byte vectors of eight columns
    const bool vec = a.N % 8 == 0 && aligned(a.y, a.ldy) && aligned(a.out, a.ldo), f32 = a.yt == BL_F32;
    // few tokens: a CTA per 32 columns and tile, its warps share the adapters;
    // else 256 columns, and a run of tiles where runs fill the GPU
    const int64_t wide = (a.N + kUpWarps * kUpCols - 1) / (kUpWarps * kUpCols);
    const int run = vec ? run_tiles(a.r <= 32 ? 2 : a.r <= 64 ? 4 : 8, f32) : 1;
    const Up kind = a.T <= kOrderTokens && tiles * wide < 2 * di->sm_count ? Up::kFew
                    : tiles * wide < run * di->sm_count                    ? Up::kTile
                                                                           : Up::kRun;
    const int64_t gx = kind == Up::kFew ? (a.N + kUpCols - 1) / kUpCols : wide;
    const int64_t gy = kind == Up::kRun ? (tiles + run - 1) / run : tiles;
    auto up = f32 ? up_kernel<true>(a.r, kind, vec) : up_kernel<false>(a.r, kind, vec);
    return cuda_status(launch(up, dim3(unsigned(gx), unsigned(std::min<int64_t>(gy, 65535))), kUpWarps * 32, s, p));
}

}  // namespace bl
