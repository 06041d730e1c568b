// adapter.cu -- low-rank adapters of many requests beside one shared
// projection: out[t] = y[t] + scale[a] up[a] (down[a] x[t]), a = index[t].
//
// Two launches, the second chained to the first (programmatic dependent
// launch): u[t] = scale[a] down[a] x[t] in fp32 to the workspace, then
// out = y + up u.  Both are bound by memory: a token brings 2 r (K + N)
// multiply-adds against 2 K + 4 N bytes, and a few tokens bring their whole
// adapters, so the products run as mma.sync m16n8k16 straight from registers
// (r columns or r terms are far too few for a tcgen05 tile) and the work is
// in keeping loads in flight:
//   - a tile is 16 tokens; the tokens' distinct adapters are found with one
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
#include <algorithm>

#include "bl_common.cuh"

namespace bl {
namespace {

constexpr int kTile = 16;                 // tokens per tile (MMA M)
constexpr int kDownWarps = 8, kUpWarps = 8;
constexpr int kUpCols = 32;               // output columns per warp

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

// The adapter of token t0 + lane (lanes 0 .. 15), -1: none; an id that does
// not exist counts as none.
__device__ __forceinline__ int tile_id(const AdapterParams &p, int64_t t0, int lane, bool report)
{
    int id = -1;
    if (lane < kTile && t0 + lane < p.T)
        id = int(ld_dep_u32(p.index + t0 + lane));
    if (id >= p.n) {
        if (report)
            atomicExch(p.status, BL_ERR_SHAPE);
        id = -1;
    }
    return id < 0 ? -1 : id;
}

// Lanes that are the first with their adapter.
__device__ __forceinline__ unsigned first_of(int id, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, id);
    return __ballot_sync(0xffffffffu, id >= 0 && lane == __ffs(same) - 1);
}

// u of one tile, one K split: the warps take the split's 32-k groups in turn
// and their sums are added through shared memory in a fixed order.
template <int NT>
__global__ void __launch_bounds__(kDownWarps * 32) adapter_down_kernel(const AdapterParams p)
{
    __shared__ float red[kDownWarps / 2][kTile][NT * 8];
    // the second launch reads y before it waits for this one, so it may begin
    // only when what came before this one is complete
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = int64_t(blockIdx.x) * kTile;
    const int way = blockIdx.y, split = blockIdx.z;
    const int groups = int(p.K / 32);
    const int k0 = int(int64_t(split) * groups / p.splits) + warp, k1 = int(int64_t(split + 1) * groups / p.splits);
    constexpr int kDeep = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;      // groups in flight
    const bool in0 = t0 + g < p.T, in1 = t0 + g + 8 < p.T;
    const __nv_bfloat16 *x0 = p.x + (t0 + g) * p.ldx + 8 * c, *x1 = x0 + 8 * p.ldx;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // all tokens' x, before their adapters are known: the rows of other
    // adapters are dropped at the end
    uint4 xa[kDeep], xb[kDeep];
    auto load_x = [&](int k) {
#pragma unroll
        for (int s = 0; s < kDeep; ++s) {
            const bool in = k + s * kDownWarps < k1;
            const int64_t at = int64_t(k + s * kDownWarps) * 32;
            xa[s] = in && in0 ? ld_dep_v4(x0 + at) : zero;
            xb[s] = in && in1 ? ld_dep_v4(x1 + at) : zero;
        }
    };
    load_x(k0);
    const bool once = k0 + kDeep * kDownWarps >= k1;          // that was all of it
    const int id = tile_id(p, t0, lane, way == 0 && split == 0);
    unsigned firsts = first_of(id, lane);
    for (int ord = 0; firsts; ++ord, firsts &= firsts - 1) {
        if (ord % p.down_ways != way)
            continue;
        const int a = __shfl_sync(0xffffffffu, id, __ffs(firsts) - 1);
        const unsigned rows = __ballot_sync(0xffffffffu, id == a);
        const __nv_bfloat16 *w = p.down + (int64_t(a) * p.r + g) * p.K + 8 * c;
        float acc[NT][4] = {};
        for (int k = k0; k < k1; k += kDeep * kDownWarps) {
            uint4 b[kDeep][NT];
            if (!once)
                load_x(k);
#pragma unroll
            for (int s = 0; s < kDeep; ++s) {
                const int64_t at = int64_t(k + s * kDownWarps) * 32;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b[s][j] = k + s * kDownWarps < k1 && j * 8 < p.r ? ld_ro_v4(w + j * 8 * p.K + at) : zero;
            }
#pragma unroll
            for (int s = 0; s < kDeep; ++s) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_bf16(acc[j], xa[s].x, xb[s].x, xa[s].y, xb[s].y, b[s][j].x, b[s][j].y);
                    mma_bf16(acc[j], xa[s].z, xb[s].z, xa[s].w, xb[s].w, b[s][j].z, b[s][j].w);
                }
            }
        }
        // sums of warps w and w + 4, then of the four pairs
        const int pair = warp & (kDownWarps / 2 - 1);
        for (int half = 1; half >= 0; --half) {
            if (warp / (kDownWarps / 2) == half) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &s = red[pair][g + 8 * (e >> 1)][8 * j + 2 * c + (e & 1)];
                        s = half ? acc[j][e] : s + acc[j][e];
                    }
                }
            }
            __syncthreads();
        }
        const float scale = p.scale ? __ldcg(p.scale + a) : 1.0f;
        for (int e = threadIdx.x; e < kTile * p.r; e += kDownWarps * 32) {
            const int row = e / p.r, j = e - row * p.r;
            if (rows >> row & 1) {
                float s = red[0][row][j];
#pragma unroll
                for (int q = 1; q < kDownWarps / 2; ++q)
                    s += red[q][row][j];
                __stcg(p.u + (int64_t(split) * p.T + t0 + row) * p.r + j, s * scale);
            }
        }
        __syncthreads();
    }
}

// Eight consecutive elements of a row, as loaded: 16-byte vectors (VEC), or one
// element after the other where rows are not aligned or end inside the eight
// (`left` of them are there).
template <bool F32, bool VEC>
struct Cols {
    uint4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const char *src, int64_t left)
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i)
                v[i] = ld_dep_v4(src + 16 * i);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = i >= left ? 0u : F32 ? ld_dep_u32(src + 4 * i) : ld_dep_u16(src + 2 * i);
            if constexpr (F32) {
                v[0] = make_uint4(w[0], w[1], w[2], w[3]);
                v[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
                v[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
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
    static __device__ __forceinline__ void store(char *dst, const float (&f)[8], int64_t left)
    {
        if constexpr (VEC && F32) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else if constexpr (VEC) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                         pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    store_y(dst, F32 ? BL_F32 : BL_BF16, i, f[i]);
        }
    }
};

// The values (a, b) as sums of TERMS bf16 values, largest first.
template <int TERMS>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&w)[TERMS])
{
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        w[i] = pack_bf16(a, b);
        a -= __uint_as_float(w[i] << 16);
        b -= __uint_as_float(w[i] & 0xffff0000u);
    }
}

// out = y + up u for runs of tiles and the columns of a CTA.  A warp has 32
// columns; WAYS = 1: the warps of a CTA lie side by side and take a run's
// tiles one after the other, every tile's y in flight from the start; WAYS = 8:
// they share 32 columns and the adapters of one tile.  y and the adapters are
// asked for while the first launch still runs.  u, the K splits' parts added
// in order, is split into its bf16 terms once per CTA, and a tile whose tokens
// share one adapter (most tiles of a prompt) keeps its operand from tile to
// tile and starts the accumulators at y (bf16 outputs; an fp32 output adds y at
// the end, since a tensor core's sums lose up to 2^-23 of y each).
template <int KB, bool F32, int WAYS, bool VEC>
__global__ void __launch_bounds__(kUpWarps * 32, 2) adapter_up_kernel(const AdapterParams p)
{
    constexpr int kTiles = WAYS == 1 ? (F32 ? 2 : 4) : 1;
    constexpr int kTokens = kTiles * kTile;
    constexpr int kTerms = F32 ? 3 : 2;
    constexpr int kPitch = 8 * KB + 4;                        // words (two ranks) per token
    __shared__ uint32_t u_s[kTerms][kTokens][kPitch];
    __shared__ int id_s[kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int way = WAYS == 1 ? 0 : warp;
    const int64_t n0 = (int64_t(blockIdx.x) * (kUpWarps / WAYS) + (WAYS == 1 ? warp : 0)) * kUpCols;
    const int64_t nc = n0 + 8 * c;                            // this lane's output columns
    const int64_t left = p.N - nc;                            // columns from there to the row's end
    const bool cols = n0 < p.N;
    constexpr int kElem = F32 ? 4 : 2;
    using Eight = Cols<F32, VEC>;
    bool waited = false;
    constexpr int kKept = KB <= 2 ? KB : 1;                   // k blocks of an adapter's operand in registers
    uint2 b[kKept][4];
    int b_of = -1;                                            // the adapter that b holds (KB <= 2)
    auto load_kb = [&](int a, int kb, uint2 (&v)[4]) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            // column g of tile x: 8 (g / 2) + 2 x + g % 2; this lane's four ranks
            const int64_t n = n0 + 8 * (g >> 1) + 2 * x + (g & 1);
            const int k = 16 * kb + 4 * c;
            v[x] = make_uint2(0, 0);
            if (k < p.r && n < p.N)
                v[x] = __ldg(reinterpret_cast<const uint2 *>(p.up + (int64_t(a) * p.N + n) * p.r + k));
        }
    };
    auto load_b = [&](int a) {
        if (KB > 2 || a == b_of)
            return;
        b_of = a;
#pragma unroll
        for (int kb = 0; kb < kKept; ++kb)
            load_kb(a, kb, b[kb]);
    };
    for (int64_t run = blockIdx.y; run * kTokens < p.T; run += gridDim.y) {
        const int64_t t0 = run * kTokens;
        const int tokens = int(min(int64_t(kTokens), p.T - t0));
        __syncthreads();                                      // the last run's u has been used
        Eight y[kTiles][2];
        {
            const char *src = static_cast<const char *>(p.y) + ((t0 + g) * p.ldy + nc) * kElem;
            const int64_t step = 8 * p.ldy * kElem;
#pragma unroll
            for (int i = 0; i < 2 * kTiles; ++i, src += step)
                if (8 * i + g < tokens && left > 0)
                    y[i / 2][i % 2].load(src, left);
        }
        if (threadIdx.x < kTokens) {
            const int id = int(threadIdx.x) < tokens ? int(ld_dep_u32(p.index + t0 + threadIdx.x)) : -1;
            id_s[threadIdx.x] = id < 0 || id >= p.n ? -1 : id;     // reported by the first launch
        }
        __syncthreads();
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
        char *dst = static_cast<char *>(p.out) + ((t0 + g) * p.ldo + nc) * kElem;
        const int64_t ostep = 8 * p.ldo * kElem;
#pragma unroll
        for (int i = 0; i < kTiles; ++i, dst += 2 * ostep) {
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
                    if (KB > 2)
                        load_kb(a, kb, b[0]);
                    uint2 (&bk)[4] = b[KB > 2 ? 0 : kb];
#pragma unroll
                    for (int q = kTerms - 1; q >= 0; --q) {
                        const uint2 ua = *reinterpret_cast<const uint2 *>(&u_s[q][16 * i + g][8 * kb + 2 * c]);
                        const uint2 ub = *reinterpret_cast<const uint2 *>(&u_s[q][16 * i + g + 8][8 * kb + 2 * c]);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_bf16(acc[x], ua.x, ub.x, ua.y, ub.y, bk[x].x, bk[x].y);
                    }
                }
            };
            const int id = lane < kTile ? id_s[16 * i + lane] : -1;
            const int valid = min(16, tokens - 16 * i), one = __shfl_sync(0xffffffffu, id, 0);
            if (!F32 && WAYS == 1 && one >= 0 && __all_sync(0xffffffffu, id == one || lane >= valid)) {
                float acc[4][4], f[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    y[i][h].floats(f);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        acc[x][2 * h] = f[2 * x];
                        acc[x][2 * h + 1] = f[2 * x + 1];
                    }
                }
                product(one, acc);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        f[2 * x] = acc[x][2 * h];
                        f[2 * x + 1] = acc[x][2 * h + 1];
                    }
                    if (g + 8 * h < valid && left > 0)
                        Eight::store(dst + h * ostep, f, left);
                }
                continue;
            }
            unsigned firsts = first_of(id, lane);
            const unsigned none = __ballot_sync(0xffffffffu, lane < valid && id < 0);
            if (way == 0) {                                   // tokens without an adapter
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((none >> (g + 8 * h) & 1) && left > 0) {
                        float f[8];
                        y[i][h].floats(f);
                        Eight::store(dst + h * ostep, f, left);
                    }
                }
            }
            for (int ord = 0; firsts; ++ord, firsts &= firsts - 1) {
                if (WAYS > 1 && ord % WAYS != way)
                    continue;
                const int a = __shfl_sync(0xffffffffu, id, __ffs(firsts) - 1);
                const unsigned rows = __ballot_sync(0xffffffffu, id == a);
                float acc[4][4] = {};
                product(a, acc);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((rows >> (g + 8 * h) & 1) && left > 0) {
                        float f[8];
                        y[i][h].floats(f);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            f[2 * x] += acc[x][2 * h];
                            f[2 * x + 1] += acc[x][2 * h + 1];
                        }
                        Eight::store(dst + h * ostep, f, left);
                    }
                }
            }
        }
    }
}

// K splits of the first launch: six CTAs per SM (a warp's groups are then in
// flight at once) while each warp still has a 32-k group (K >= 64; T is all the workspace's size may depend on, so
// the splits go by the tokens and the launch takes no more than K allows).
int max_splits(int64_t T, int sms)
{
    const int64_t tiles = (T + kTile - 1) / kTile;
    return int(std::clamp<int64_t>(6 * sms / tiles, 1, 32));
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

template <bool F32, int WAYS, bool VEC>
auto up_kernel(int r) -> void (*)(AdapterParams)
{
    return r <= 16   ? adapter_up_kernel<1, F32, WAYS, VEC>
           : r <= 32 ? adapter_up_kernel<2, F32, WAYS, VEC>
           : r <= 64 ? adapter_up_kernel<4, F32, WAYS, VEC>
                     : adapter_up_kernel<8, F32, WAYS, VEC>;
}

template <bool F32>
auto up_kernel(int r, bool few, bool vec) -> void (*)(AdapterParams)
{
    return few ? (vec ? up_kernel<F32, 8, true>(r) : up_kernel<F32, 8, false>(r))
               : (vec ? up_kernel<F32, 1, true>(r) : up_kernel<F32, 1, false>(r));
}

}  // namespace

size_t adapter_workspace_bytes(int64_t T, int r)
{
    const DeviceInfo *di = device_info();
    return di ? size_t(max_splits(T, di->sm_count)) * size_t(T) * size_t(r) * sizeof(float) : 0;
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
    p.splits = int(std::clamp<int64_t>(a.K / 32 / kDownWarps, 1, max_splits(a.T, di->sm_count)));
    p.status = di->status;
    // a tile's adapters go to CTAs of their own while tiles alone do not fill the GPU
    p.down_ways = int(std::clamp<int64_t>(di->sm_count / tiles, 1, std::min<int64_t>({kTile, a.n, a.T})));
    auto down = a.r <= 8    ? adapter_down_kernel<1>
                : a.r <= 16 ? adapter_down_kernel<2>
                : a.r <= 32 ? adapter_down_kernel<4>
                : a.r <= 64 ? adapter_down_kernel<8>
                            : adapter_down_kernel<16>;
    const dim3 dgrid(unsigned(tiles), unsigned(p.down_ways), unsigned(p.splits));
    int st = cuda_status(launch(down, dgrid, kDownWarps * 32, s, p));
    if (st)
        return st;
    // few tokens: a CTA per 32 columns and 16 tokens, its warps share the adapters
    const bool few = tiles * ((a.N + 8 * kUpCols - 1) / (8 * kUpCols)) < 2 * di->sm_count;
    const int cols = few ? kUpCols : kUpWarps * kUpCols, tokens = kTile * (few ? 1 : a.yt == BL_F32 ? 2 : 4);
    const int64_t gx = (a.N + cols - 1) / cols, gy = (a.T + tokens - 1) / tokens;
    // rows of whole 16-byte vectors of eight columns
    const bool vec = a.N % 8 == 0 && aligned(a.y, a.ldy) && aligned(a.out, a.ldo);
    auto up = a.yt == BL_F32 ? up_kernel<true>(a.r, few, vec) : up_kernel<false>(a.r, few, vec);
    return cuda_status(launch(up, dim3(unsigned(gx), unsigned(std::min<int64_t>(gy, 65535))), kUpWarps * 32, s, p));
}

}  // namespace bl
