// qk_norm_rope.cu -- RMS norm of query and key heads, rotation by the token's
// position and the write of keys and values to their cache rows, for many
// tokens in one pass.
//
// "bit-floor" README, section "What's inside" (RMSNorm; RoPE on queries and
// keys before attention).  Per head x of 128 values (all in fp32):
//   r = 1 / sqrt(mean x^2 + eps),  h = (x * r) * g      (only with a gain)
//   (a, b) <- (a c - b s, a s + b c)                     (c, s) of the position
// rounded once to bf16.  The rotation's operations and their order are those
// of attention.cu, so a prompt's cache rows equal the rows that its tokens
// would get one at a time.
//
// Memory-bound: every element is read once and written once.  Eight lanes
// take a head, each with dimensions 8c .. 8c + 7 and 64 + 8c .. 64 + 8c + 7, so
// that every load and store of bf16 is 16 bytes a lane and 128 contiguous
// bytes a head, and both kinds of pairs ((2i, 2i + 1) and (i, i + 64)) are
// inside one lane; the mean square is a sum over three shuffles.  A warp takes
// four heads at a time of one token, whose angles stay in registers, and asks
// for several steps' heads before it knows the token's position.
#include <algorithm>

#include "bl_common.cuh"

namespace bl {
namespace {

constexpr int kHD = 128;
constexpr int kRopeThreads = 256;
constexpr int kHeadLanes = 8;

struct RopeParams {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    __nv_bfloat16 *qo, *ko, *vo;
    int64_t qo_row, qo_head, ko_row, ko_head, vo_row, vo_head;
    int T, H, Hkv, heads;          // heads: H + Hkv (+ Hkv with values)
    int parts, steps;              // warps per token, steps of four heads each takes
    const int32_t *positions;
    const float2 *table;
    int64_t table_rows;
    const void *q_gain, *k_gain;
    int gt;
    float eps;
    const int32_t *slots;
    int64_t out_rows;
    int *status;
};

// Eight gain values (fp32 or bf16).
__device__ __forceinline__ void gain8(const void *g, int gt, int at, float f[8])
{
    if (gt == BL_BF16)
        load8<BL_BF16>(g, at, f);
    else
        load8<BL_F32>(g, at, f);
}

// Eight elements as loaded: one 16-byte vector of bf16, two of fp32.
template <int XT>
struct Raw8 {
    uint4 v[XT == BL_BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *base, int64_t at)
    {
        if constexpr (XT == BL_BF16) {
            v[0] = ld_dep_v4(static_cast<const __nv_bfloat16 *>(base) + at);
        } else {
            v[0] = ld_dep_v4(static_cast<const float *>(base) + at);
            v[1] = ld_dep_v4(static_cast<const float *>(base) + at + 4);
        }
    }
    __device__ __forceinline__ void floats(float f[8]) const
    {
        if constexpr (XT == BL_BF16) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __uint_as_float(w[i]);
        }
    }
};

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float f[8])
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ void rotate(float &a, float &b, float2 cs)
{
    const float r0 = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
    const float r1 = __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
    a = r0;
    b = r1;
}

template <int XT, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 2) qk_norm_rope_kernel(const RopeParams p)
{
    constexpr int kAhead = XT == BL_BF16 ? 3 : 2;        // steps whose heads are in flight
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t item = (int64_t(blockIdx.x) * kRopeThreads + threadIdx.x) / 32;
    const int64_t t = item / p.parts;
    if (t >= p.T)
        return;
    const int lane = threadIdx.x & 31, c = lane % kHeadLanes;
    const int first = int(item - t * p.parts) * p.steps * 4 + lane / kHeadLanes;     // this lane's first head
    const int last = min(p.heads, (int(item - t * p.parts) + 1) * p.steps * 4);
    Raw8<XT> lo[kAhead], hi[kAhead];
    auto load = [&](int h, Raw8<XT> &a, Raw8<XT> &b) {
        if (h >= last)
            return;
        const void *src = h < p.H ? p.q : h < p.H + p.Hkv ? p.k : p.v;
        const int64_t at = h < p.H            ? t * p.q_row + h * p.q_head
                           : h < p.H + p.Hkv ? t * p.k_row + (h - p.H) * p.k_head
                                              : t * p.v_row + (h - p.H - p.Hkv) * p.v_head;
        a.load(src, at + 8 * c);
        b.load(src, at + 64 + 8 * c);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        load(first + 4 * u, lo[u], hi[u]);
    const int64_t pos = int32_t(ld_dep_u32(p.positions + t));
    int64_t row = p.slots ? int32_t(ld_dep_u32(p.slots + t)) : t;
    const bool bad_pos = pos < 0 || pos >= p.table_rows, bad_row = p.slots && row >= p.out_rows;
    if (bad_pos || bad_row) {
        if (lane == 0)
            atomicExch(p.status, BL_ERR_SHAPE);
        if (bad_pos)
            return;
        row = -1;
    }
    // (cos, sin) of this lane's pairs: 8c .. 8c + 7, or 4c .. 4c + 3 and 32 + 4c .. 32 + 4c + 3
    const float2 *tab = p.table + pos * (kHD / 2);
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        cs[i] = __ldg(tab + (HALVES ? 8 * c + i : i < 4 ? 4 * c + i : 32 + 4 * c + i - 4));
    // gains of the kind of head (0: query, 1: key) that was taken last
    float ga[8], gb[8];
    int kind = -1;
    for (int h0 = first; h0 - lane / kHeadLanes < last; h0 += 4 * kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + 4 * u;
            if (h - lane / kHeadLanes >= last)
                break;
            float a[8], b[8];
            lo[u].floats(a);
            hi[u].floats(b);
            const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hkv;
            const void *gain = is_q ? p.q_gain : is_k ? p.k_gain : nullptr;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
#pragma unroll
            for (int o = kHeadLanes / 2; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            load(h + 4 * kAhead, lo[u], hi[u]);
            if (h >= last || (!is_q && row < 0))
                continue;
            if (gain) {
                if (kind != int(is_k)) {
                    kind = is_k;
                    gain8(gain, p.gt, 8 * c, ga);
                    gain8(gain, p.gt, 64 + 8 * c, gb);
                }
                // fp32 to 2^-22; the result rounds at 2^-8
                const float r = rsqrtf(fmaf(s, 1.0f / kHD, p.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = a[i] * r * ga[i];
                    b[i] = b[i] * r * gb[i];
                }
            }
            if (is_q || is_k) {
                if (HALVES) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        rotate(a[i], b[i], cs[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        rotate(a[2 * i], a[2 * i + 1], cs[i]);
                        rotate(b[2 * i], b[2 * i + 1], cs[4 + i]);
                    }
                }
            }
            __nv_bfloat16 *dst = is_q   ? p.qo + t * p.qo_row + h * p.qo_head
                                 : is_k ? p.ko + row * p.ko_row + (h - p.H) * p.ko_head
                                        : p.vo + row * p.vo_row + (h - p.H - p.Hkv) * p.vo_head;
            *reinterpret_cast<uint4 *>(dst + 8 * c) = pack8(a);
            *reinterpret_cast<uint4 *>(dst + 64 + 8 * c) = pack8(b);
        }
    }
}

}  // namespace

int launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t s)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return BL_ERR_CUDA;
    RopeParams p{};
    p.q = a.q.data;
    p.q_row = a.q.row_stride;
    p.q_head = a.q.head_stride;
    p.k = a.k.data;
    p.k_row = a.k.row_stride;
    p.k_head = a.k.head_stride;
    p.v = a.v.data;
    p.v_row = a.v.row_stride;
    p.v_head = a.v.head_stride;
    p.qo = static_cast<__nv_bfloat16 *>(a.q_out.data);
    p.qo_row = a.q_out.row_stride;
    p.qo_head = a.q_out.head_stride;
    p.ko = static_cast<__nv_bfloat16 *>(a.k_out.data);
    p.ko_row = a.k_out.row_stride;
    p.ko_head = a.k_out.head_stride;
    p.vo = static_cast<__nv_bfloat16 *>(a.v_out.data);
    p.vo_row = a.v_out.row_stride;
    p.vo_head = a.v_out.head_stride;
    p.T = int(a.q.rows);
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.heads = a.H + a.Hkv + (a.v.data ? a.Hkv : 0);
    p.positions = a.positions;
    p.table = reinterpret_cast<const float2 *>(a.table);
    p.table_rows = a.table_rows;
    p.q_gain = a.q_gain;
    p.k_gain = a.k_gain;
    p.gt = a.gt;
    p.eps = a.eps;
    p.slots = a.slots;
    p.out_rows = a.k_out.rows;
    p.status = di->status;
    // a token's heads go to one warp where the tokens fill the GPU (two
    // CTAs' warps per SM and more), else to as many as there are steps
    const int all = (p.heads + 3) / 4;
    p.parts = int(std::clamp<int64_t>(int64_t(di->sm_count) * 16 / p.T, 1, all));
    p.steps = (all + p.parts - 1) / p.parts;
    p.parts = (all + p.steps - 1) / p.steps;
    const int64_t blocks = (int64_t(p.T) * p.parts * 32 + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7fffffff)
        return BL_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    // the kernel reads and writes nothing before what came before it is complete
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool halves = a.flags & BL_FLAG_ROPE_HALVES;
    auto kernel = a.xt == BL_BF16 ? (halves ? qk_norm_rope_kernel<BL_BF16, true> : qk_norm_rope_kernel<BL_BF16, false>)
                                  : (halves ? qk_norm_rope_kernel<BL_F32, true> : qk_norm_rope_kernel<BL_F32, false>);
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

}  // namespace bl
