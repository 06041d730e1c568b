// attention_prefill.cu -- causal attention of packed sequences with grouped
// heads.  One warp per (query, head), keys one after the other with a running
// maximum m and sum l of the softmax:
//   m' = max(m, s_j), l <- l e^(m - m') + e^(s_j - m'), o <- o e^(m - m') + e^(s_j - m') V[j]
#include "bl_common.cuh"

namespace bl {
namespace {

constexpr int kHD = 128;

struct PrefillParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
    const int32_t *cu_q, *cu_k;
    int batch, H, group;
    int64_t Tq, Tk;
    float scale;
    int *status;
};

__device__ __forceinline__ void load4(const __nv_bfloat16 *src, float f[4])
{
    const uint2 w = *reinterpret_cast<const uint2 *>(src);
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xffff0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xffff0000u);
}

__global__ void __launch_bounds__(128) prefill_kernel(const PrefillParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += 128)
            if (p.cu_q[b] < 0 || p.cu_q[b + 1] < p.cu_q[b] || int64_t(p.cu_q[b + 1]) > p.Tq || p.cu_k[b] < 0 ||
                p.cu_k[b + 1] < p.cu_k[b] || int64_t(p.cu_k[b + 1]) > p.Tk)
                atomicExch(p.status, BL_ERR_SHAPE);
    const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / p.H;
    const int h = int(item - t * p.H);
    if (t >= p.Tq)
        return;
    int64_t q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    for (int b = 0; b < p.batch && !(q0 <= t && t < q1); ++b) {
        q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
        if (q0 < 0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk)
            q1 = q0;        // reported above
    }
    if (t < q0 || t >= q1)
        return;
    const int64_t seen = (k1 - k0) - (q1 - 1 - t);      // keys below this are visible
    float q[4], o[4] = {};
    load4(p.q + t * p.q_row + h * p.q_head + 4 * lane, q);
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j < seen; ++j) {
        float k[4], v[4];
        load4(p.k + (k0 + j) * p.k_row + h / p.group * p.k_head + 4 * lane, k);
        load4(p.v + (k0 + j) * p.v_row + h / p.group * p.v_head + 4 * lane, v);
        const float s = p.scale * warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
        const float m1 = fmaxf(m, s), f = expf(m - m1), e = expf(s - m1);
        m = m1;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = o[i] * f + e * v[i];
    }
    __nv_bfloat16 *dst = p.out + t * p.o_row + h * p.o_head + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        dst[i] = __float2bfloat16_rn(seen > 0 ? o[i] / l : 0.0f);
}

}  // namespace

size_t attention_prefill_workspace_bytes(int, int) { return 16; }

int launch_attention_prefill(const PrefillArgs &a, cudaStream_t s)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return BL_ERR_CUDA;
    const PrefillParams p{static_cast<const __nv_bfloat16 *>(a.q.data), static_cast<const __nv_bfloat16 *>(a.k.data),
                          static_cast<const __nv_bfloat16 *>(a.v.data), static_cast<__nv_bfloat16 *>(a.out.data),
                          a.q.row_stride, a.q.head_stride, a.k.row_stride, a.k.head_stride, a.v.row_stride,
                          a.v.head_stride, a.out.row_stride, a.out.head_stride, a.cu_q, a.cu_k, a.batch, a.H,
                          a.H / a.Hkv, a.q.rows, a.k.rows, a.scale, di->status};
    const int64_t blocks = (p.Tq * p.H + 3) / 4;
    if (blocks > 0x7fffffff)
        return BL_ERR_SHAPE;
    prefill_kernel<<<unsigned(blocks), 128, 0, s>>>(p);
    return launch_status();
}

}  // namespace bl
