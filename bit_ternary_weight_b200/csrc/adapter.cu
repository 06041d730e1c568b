// adapter.cu -- low-rank adapters of many requests beside one projection:
//   u[t] = down[a] x[t] (fp32, workspace), out[t] = y[t] + scale[a] up[a] u[t].
// One warp per (token, rank) of u, one thread per output.
#include "bl_common.cuh"

namespace bl {
namespace {

__global__ void __launch_bounds__(128) adapter_down_kernel(const AdapterArgs a, float *u, int *status)
{
    const int64_t item = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = item / a.r;
    const int j = int(item - t * a.r);
    if (t >= a.T)
        return;
    const int id = a.index[t];
    if (id < 0)
        return;
    if (id >= a.n) {
        if (lane == 0)
            atomicExch(status, BL_ERR_SHAPE);
        return;
    }
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + t * a.ldx;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(a.down) + (int64_t(id) * a.r + j) * a.K;
    float s = 0.0f;
    for (int64_t k = lane; k < a.K; k += 32)
        s = fmaf(__bfloat162float(x[k]), __bfloat162float(w[k]), s);
    s = warp_sum(s);
    if (lane == 0)
        u[t * a.r + j] = a.scale ? s * a.scale[id] : s;
}

__global__ void __launch_bounds__(128) adapter_up_kernel(const AdapterArgs a, const float *u)
{
    const int64_t n = int64_t(blockIdx.x) * 128 + threadIdx.x;
    if (n >= a.N)
        return;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const int id = a.index[t];
        float v = a.yt == BL_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.y)[t * a.ldy + n])
                                  : static_cast<const float *>(a.y)[t * a.ldy + n];
        if (id >= 0 && id < a.n) {
            const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(a.up) + (int64_t(id) * a.N + n) * a.r;
            float s = 0.0f;
            for (int j = 0; j < a.r; ++j)
                s = fmaf(u[t * a.r + j], __bfloat162float(w[j]), s);
            v += s;
        }
        store_y(a.out, a.yt, t * a.ldo + n, v);
    }
}

}  // namespace

size_t adapter_workspace_bytes(int64_t T, int r) { return size_t(T) * size_t(r) * sizeof(float); }

int launch_adapter_add(const AdapterArgs &a, cudaStream_t s)
{
    const DeviceInfo *di = device_info();
    if (!di)
        return BL_ERR_CUDA;
    float *u = static_cast<float *>(a.ws);
    const int64_t blocks = (a.T * a.r + 3) / 4;
    if (blocks > 0x7fffffff)
        return BL_ERR_SHAPE;
    adapter_down_kernel<<<unsigned(blocks), 128, 0, s>>>(a, u, di->status);
    int st = launch_status();
    if (st)
        return st;
    const dim3 grid(unsigned((a.N + 127) / 128), unsigned(a.T < 4096 ? a.T : 4096));
    adapter_up_kernel<<<grid, 128, 0, s>>>(a, u);
    return launch_status();
}

}  // namespace bl
