// qk_norm_rope.cu -- RMS norm of query and key heads, rotation by the token's
// position and the write of keys and values to their cache rows, for many
// tokens in one pass.
//
// "bit-floor" README, section "What's inside" (RMSNorm; RoPE on queries and
// keys before attention).  Per head x of 128 values (all in fp32):
//   r = 1 / sqrt(mean x^2 + eps),  h = (x * r) * g      (only with a gain)
//   (a, b) <- (a c - b s, a s + b c)                     (c, s) of the position
// rounded once to bf16.  Without a gain the rotation's operations and their
// order are those of attention.cu, so a prompt's cache rows equal the rows that
// its tokens would get one at a time; with one, gains are folded into the
// angles and r is applied last (below).
//
// Memory-bound: every element is read once and written once, so the design is
// about bytes in flight.  A warp takes the heads of a token (or a part of
// them), which one bulk copy per head, each issued by a lane, brings to a slot
// of the warp's in shared memory, two slots a warp, so that one token arrives
// while the other is worked on.  An 8192-token prompt of 20 + 5 + 5 heads
// (126 MB): 32 us, 3.9 TB/s; with loads to registers, three steps of four heads
// ahead, 39 us.  What bounds it is the arithmetic's latency at 12 warps an SM:
// without any store it still takes 30 us.  (8 warps of three slots: 36 us.)
// 1283 tokens in fp32 (30 MB): 8.3 us; a slot holds 16 fp32 heads, so a token is
// two items, 2566 on 1776 warps, and most warps have no second one.
// Eight lanes take a head from the slot, each
// with dimensions 8c .. 8c + 7 and 64 + 8c .. 64 + 8c + 7, so that every access
// is 16 bytes a lane and both kinds of pairs ((2i, 2i + 1) and (i, i + 64)) are
// inside one lane; the mean square is a sum over three shuffles.  Two pairs go
// through each arithmetic instruction (packed fp32), and what multiplies a
// value is made once for a token's queries and once for its keys: with a
// gain, x r g c is r (x (g c)).
#include <algorithm>

#include "bl_common.cuh"

namespace bl {
namespace {

constexpr int kHD = 128;
constexpr int kRopeWarps = 12;
constexpr int kHeadLanes = 8;
constexpr int kRopeSlots = 2;             // items on their way per warp
constexpr int kSlotBytes = 8192;          // 32 heads of bf16, 16 of fp32

struct RopeParams {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    __nv_bfloat16 *qo, *ko, *vo;
    int64_t qo_row, qo_head, ko_row, ko_head, vo_row, vo_head;
    int T, H, Hkv, heads;          // heads: H + Hkv (+ Hkv with values)
    int parts, part;               // parts of a token's heads, heads of each
    int64_t items;                 // T * parts
    bool runs;                     // the heads of a token's queries (keys, values) are contiguous
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

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two fp32 values in one register pair, and what is done to both at once.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ void get(float &lo, float &hi) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    }
};
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// A lane's sixteen elements of a head: 8c .. 8c + 7 and 64 + 8c .. 64 + 8c + 7.
template <int XT>
struct Raw {
    static constexpr int kVecs = XT == BL_BF16 ? 1 : 2;
    uint4 v[2][kVecs];
    __device__ __forceinline__ void load(const unsigned char *head, int c)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                v[h][i] = *reinterpret_cast<const uint4 *>(head + (h * 64 + 8 * c) * (XT == BL_BF16 ? 2 : 4) + 16 * i);
    }
    // Elements e and e + 1 (e even) of half h.
    __device__ __forceinline__ void two(int h, int e, float &x, float &y) const
    {
        const uint4 &q = v[h][XT == BL_BF16 ? 0 : e / 4];
        if constexpr (XT == BL_BF16) {
            const uint32_t w = e == 0 ? q.x : e == 2 ? q.y : e == 4 ? q.z : q.w;
            x = __uint_as_float(w << 16);
            y = __uint_as_float(w & 0xffff0000u);
        } else {
            x = __uint_as_float(e % 4 ? q.z : q.x);
            y = __uint_as_float(e % 4 ? q.w : q.y);
        }
    }
    // Pairs (a, b) number 2j and 2j + 1 of the lane's eight.
    template <bool HALVES>
    __device__ __forceinline__ void pairs(int j, F2 &a, F2 &b) const
    {
        float x0, x1, y0, y1;
        if (HALVES) {
            two(0, 2 * j, x0, x1);
            two(1, 2 * j, y0, y1);
            a = F2(x0, x1);
            b = F2(y0, y1);
        } else {
            two(j / 2, 4 * (j % 2), x0, x1);
            two(j / 2, 4 * (j % 2) + 2, y0, y1);
            a = F2(x0, y0);
            b = F2(x1, y1);
        }
    }
};

// Norm (NORM) and rotation of every fourth of `heads` heads, from the group's
// first at `src` on, eight lanes a head.
//   (a, b) -> (a c1 + b s1, a s2 + b c2) with c1 = g_a c, s1 = -g_b s, s2 = g_a s,
//   c2 = g_b c, pairs two by two (g = 1 without a norm)
template <int XT, bool HALVES, bool NORM>
__device__ __forceinline__ void rotate_heads(const unsigned char *src, __nv_bfloat16 *dst, int64_t ohead, int heads,
                                             int group, int c, const float2 (&cs)[8], const void *gain, int gt, float eps)
{
    constexpr int kHeadBytes = kHD * (XT == BL_BF16 ? 2 : 4);
    F2 c1[4], s1[4], s2[4], c2[4];
    float gl[8], gh[8];
    if (NORM) {
        gain8(gain, gt, 8 * c, gl);
        gain8(gain, gt, 64 + 8 * c, gh);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = cs[2 * j], y = cs[2 * j + 1];
        c1[j] = c2[j] = F2(x.x, y.x);
        s2[j] = F2(x.y, y.y);
        s1[j] = F2(-x.y, -y.y);
        if (NORM) {
            const float *g = j < 2 ? gl : gh;
            const F2 ga = HALVES ? F2(gl[2 * j], gl[2 * j + 1]) : F2(g[4 * (j % 2)], g[4 * (j % 2) + 2]);
            const F2 gb = HALVES ? F2(gh[2 * j], gh[2 * j + 1]) : F2(g[4 * (j % 2) + 1], g[4 * (j % 2) + 3]);
            c1[j] = mul(c1[j], ga);
            s2[j] = mul(s2[j], ga);
            s1[j] = mul(s1[j], gb);
            c2[j] = mul(c2[j], gb);
        }
    }
    const int64_t ostep = 4 * ohead;
#pragma unroll 2
    for (int more = heads; more > 0; more -= 4, src += 4 * kHeadBytes, dst += ostep) {
        // a group behind the last head computes on what lies there and stores nothing
        Raw<XT> x;
        x.load(src, c);
        F2 a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.template pairs<HALVES>(j, a[j], b[j]);
        F2 r2;
        if (NORM) {
            F2 sum = mul(a[0], a[0]), sum1 = mul(b[0], b[0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) {
                sum = fma(a[j], a[j], sum);
                sum1 = fma(b[j], b[j], sum1);
            }
            float s0, s;
            add(sum, sum1).get(s0, s);
            s += s0;
#pragma unroll
            for (int o = kHeadLanes / 2; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            // fp32 to 2^-22; the result rounds at 2^-8
            s = rsqrtf(fmaf(s, 1.0f / kHD, eps));
            r2 = F2(s, s);
        }
        uint32_t w[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            F2 o0, o1;
            if (NORM) {
                o0 = mul(fma(a[j], c1[j], mul(b[j], s1[j])), r2);
                o1 = mul(fma(a[j], s2[j], mul(b[j], c2[j])), r2);
            } else {
                o0 = add(mul(a[j], c1[j]), mul(b[j], s1[j]));
                o1 = add(mul(a[j], s2[j]), mul(b[j], c2[j]));
            }
            float a0, a1, b0, b1;
            o0.get(a0, a1);
            o1.get(b0, b1);
            if (HALVES) {
                w[0][j] = pack2(a0, a1);
                w[1][j] = pack2(b0, b1);
            } else {
                w[j / 2][2 * (j % 2)] = pack2(a0, b0);
                w[j / 2][2 * (j % 2) + 1] = pack2(a1, b1);
            }
        }
        if (more > group) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
            *reinterpret_cast<uint4 *>(dst + 64) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
        }
    }
}

struct RopeSmem {
    alignas(128) unsigned char slot[kRopeWarps][kRopeSlots][kSlotBytes];
    unsigned char behind[3 * 4 * kHD];   // what the groups behind the last head of the last slot read
    uint64_t full[kRopeWarps][kRopeSlots];
    int abort_flag;
};

template <int XT, bool HALVES>
__global__ void __launch_bounds__(kRopeWarps * 32, 1) qk_norm_rope_kernel(const RopeParams p)
{
    extern __shared__ __align__(128) unsigned char rope_raw[];
    RopeSmem &sm = *reinterpret_cast<RopeSmem *>(rope_raw);
    constexpr uint32_t kHeadBytes = kHD * (XT == BL_BF16 ? 2 : 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kHeadLanes;
    if (lane == 0) {
        for (int i = 0; i < kRopeSlots; ++i)
            mbar_init(smem_u32(&sm.full[warp][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (warp == 0)
            sm.abort_flag = 0;
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t stride = int64_t(gridDim.x) * kRopeWarps;
    const int64_t item0 = int64_t(blockIdx.x) * kRopeWarps + warp;
    auto token = [&](int64_t item) { return p.parts == 1 ? item : item / p.parts; };
    // the heads of an item to slot i
    auto fetch = [&](int64_t item, int i) {
        if (item >= p.items)
            return;
        const int64_t t = token(item);
        const int h0 = int(item - t * p.parts) * p.part, n = min(p.part, p.heads - h0);
        const uint32_t bar = smem_u32(&sm.full[warp][i]);
        if (lane == 0)
            mbar_arrive_tx(bar, n * kHeadBytes);
        __syncwarp();
        // heads that lie one behind the other in one copy: lane 0, 1, 2 for
        // queries, keys, values; else a head per lane
        const int h = p.runs ? max(h0, lane == 0 ? 0 : lane == 1 ? p.H : p.H + p.Hkv) : h0 + lane;
        const int stop = min(h0 + n, !p.runs ? h + 1 : lane == 0 ? p.H : lane == 1 ? p.H + p.Hkv : p.heads);
        if (h < stop && (!p.runs || lane < 3)) {
            const void *src = h < p.H ? p.q : h < p.H + p.Hkv ? p.k : p.v;
            const int64_t at = h < p.H            ? t * p.q_row + h * p.q_head
                               : h < p.H + p.Hkv ? t * p.k_row + (h - p.H) * p.k_head
                                                  : t * p.v_row + (h - p.H - p.Hkv) * p.v_head;
            bulk_load(smem_u32(&sm.slot[warp][i][(h - h0) * kHeadBytes]),
                      static_cast<const char *>(src) + at * (XT == BL_BF16 ? 2 : 4), (stop - h) * kHeadBytes, bar);
        }
    };
    auto position = [&](int64_t item) { return item < p.items ? int(ld_dep_u32(p.positions + token(item))) : 0; };
    auto slot_row = [&](int64_t item) {
        return item < p.items && p.slots ? int(ld_dep_u32(p.slots + token(item))) : 0;
    };
    for (int i = 0; i < kRopeSlots; ++i)
        fetch(item0 + i * stride, i);
    int pos = position(item0), srow = slot_row(item0);
    int pos1 = position(item0 + stride), srow1 = slot_row(item0 + stride);
    uint32_t phase = 0;
    int slot = 0;
    for (int64_t item = item0; item < p.items; item += stride) {
        const int pos2 = position(item + 2 * stride), srow2 = slot_row(item + 2 * stride);
        const int64_t t = token(item);
        const int h0 = int(item - t * p.parts) * p.part, end = min(h0 + p.part, p.heads);
        int64_t row = p.slots ? srow : t;
        const bool bad_pos = pos < 0 || pos >= p.table_rows, bad_row = p.slots && row >= p.out_rows;
        if ((bad_pos || bad_row) && lane == 0)
            atomicExch(p.status, BL_ERR_SHAPE);
        if (bad_row)
            row = -1;
        // (cos, sin) of the lane's pairs, on their way while the heads arrive:
        // pairs 8c .. 8c + 7, or 4c .. 4c + 3 and 32 + 4c .. 32 + 4c + 3
        float2 cs[8];
        const float2 *tab = p.table + int64_t(bad_pos ? 0 : pos) * (kHD / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            cs[j] = __ldg(tab + (HALVES ? 8 * c : j < 4 ? 4 * c : 32 + 4 * c - 4) + j);
        if (!mbar_wait_fast(smem_u32(&sm.full[warp][slot]), phase, &sm.abort_flag, p.status)) {
            // given up: the copies on their way have landed before the CTA exits
            volatile int no_abort = 0;
            for (int i = 0; i < kRopeSlots && item + i * stride < p.items; ++i) {
                mbar_wait(smem_u32(&sm.full[warp][slot]), phase, &no_abort, p.status, 100000000ull);
                phase ^= slot == kRopeSlots - 1;
                slot = slot == kRopeSlots - 1 ? 0 : slot + 1;
            }
            break;
        }
        const int group = lane / kHeadLanes;
#pragma unroll 1
        for (int kind = 0; kind < 3; ++kind) {
            // this item's queries, keys or values: heads lo .. hi - 1
            const int begin = kind == 0 ? 0 : kind == 1 ? p.H : p.H + p.Hkv;
            const int lo = max(h0, begin), hi = min(end, kind == 0 ? p.H : kind == 1 ? p.H + p.Hkv : p.heads);
            if (lo >= hi || bad_pos || (kind > 0 && row < 0))
                continue;
            const int64_t ohead = kind == 0 ? p.qo_head : kind == 1 ? p.ko_head : p.vo_head;
            __nv_bfloat16 *dst = (kind == 0   ? p.qo + t * p.qo_row
                                  : kind == 1 ? p.ko + row * p.ko_row
                                              : p.vo + row * p.vo_row) + (lo - begin + group) * ohead + 8 * c;
            const unsigned char *src = &sm.slot[warp][slot][(lo - h0 + group) * kHeadBytes];
            if (kind == 2) {
                for (int h = lo + group; h < hi; h += 4, src += 4 * kHeadBytes, dst += 4 * ohead) {
                    Raw<XT> x;
                    x.load(src, c);
                    if constexpr (XT == BL_BF16) {
                        *reinterpret_cast<uint4 *>(dst) = x.v[0][0];
                        *reinterpret_cast<uint4 *>(dst + 64) = x.v[1][0];
                    } else {
                        uint32_t w[2][4];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float a, b;
                            x.two(e / 4, 2 * (e % 4), a, b);
                            w[e / 4][e % 4] = pack2(a, b);
                        }
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
                        *reinterpret_cast<uint4 *>(dst + 64) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
                    }
                }
                continue;
            }
            const void *gain = kind ? p.k_gain : p.q_gain;
            if (gain)
                rotate_heads<XT, HALVES, true>(src, dst, ohead, hi - lo, group, c, cs, gain, p.gt, p.eps);
            else
                rotate_heads<XT, HALVES, false>(src, dst, ohead, hi - lo, group, c, cs, nullptr, 0, 0.0f);
        }
        __syncwarp();       // every lane has taken its part of the slot
        fetch(item + kRopeSlots * stride, slot);
        if (++slot == kRopeSlots) {
            slot = 0;
            phase ^= 1u;
        }
        pos = pos1;
        srow = srow1;
        pos1 = pos2;
        srow1 = srow2;
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
    // a token's heads go to as many warps as there are for it, four heads a
    // warp or more, and as a slot needs them to
    const int64_t warps = int64_t(di->sm_count) * kRopeWarps;
    const int room = kSlotBytes / (kHD * (a.xt == BL_BF16 ? 2 : 4)), fours = (p.heads + 3) / 4;
    const int64_t want = std::clamp<int64_t>(warps / p.T, 1, fours);
    p.part = std::min(room, int((fours + want - 1) / want) * 4);
    p.parts = (p.heads + p.part - 1) / p.part;
    p.items = int64_t(p.T) * p.parts;
    auto run = [](const bitlinear_heads &h, int heads) { return heads == 1 || h.head_stride == kHD; };
    p.runs = run(a.q, a.H) && run(a.k, a.Hkv) && (!a.v.data || run(a.v, a.Hkv));
    const int64_t blocks = std::min<int64_t>(di->sm_count, (p.items + kRopeWarps - 1) / kRopeWarps);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kRopeWarps * 32);
    cfg.dynamicSmemBytes = sizeof(RopeSmem);
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
    int per_sm = 0;
    const int st = occupancy(reinterpret_cast<const void *>(kernel), kRopeWarps * 32, sizeof(RopeSmem), &per_sm);
    if (st)
        return st;
    if (per_sm < 1)
        return BL_ERR_UNSUPPORTED;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

}  // namespace bl
