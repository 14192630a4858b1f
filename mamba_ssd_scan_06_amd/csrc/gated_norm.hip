// RMS norm with a gate over each of a row's ngroups parts:
//     v = x silu(z), out = v rsqrt(mean v^2 + eps) weight      (gate first), or
//     out = x rsqrt(mean x^2 + eps) weight silu(z)             (norm first).
// One workgroup per part of a row: the sum of squares in fp32, then the
// scaled values.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(NormParams p) {
    __shared__ float part[kThreads / kWave];
    const int64_t parts = p.rows * p.ngroups;
    for (int64_t k = blockIdx.x; k < parts; k += gridDim.x) {
        const int64_t row = k / p.ngroups;
        const int c0 = (int)(k - row * p.ngroups) * p.group_dim;
        const int64_t b = row / p.seqlen, t = row - b * p.seqlen;
        const T *x = reinterpret_cast<const T *>(p.x) + b * p.x_bs + t * p.x_ts + c0;
        const T *z = p.z ? reinterpret_cast<const T *>(p.z) + b * p.z_bs + t * p.z_ts + c0 : nullptr;
        T *out = reinterpret_cast<T *>(p.out) + row * p.dim + c0;
        float sum = 0.0f;
        for (int i = threadIdx.x; i < p.group_dim; i += kThreads) {
            float v = to_f32(x[i]);
            if (z && !p.norm_before_gate) v *= silu(to_f32(z[i]));
            sum = fmaf(v, v, sum);
        }
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < kThreads / kWave; ++w) sum += part[w];
        __syncthreads();
        const float scale = 1.0f / sqrtf(sum / (float)p.group_dim + p.eps);
        for (int i = threadIdx.x; i < p.group_dim; i += kThreads) {
            float v = to_f32(x[i]) * scale;
            if (p.weight) v *= p.weight[c0 + i];
            if (z) v *= silu(to_f32(z[i]));
            out[i] = from_f32<T>(v);
        }
    }
}

template <typename T>
hipError_t run(const NormParams &p, hipStream_t stream) {
    const unsigned grid = (unsigned)std::min<int64_t>(p.rows * p.ngroups, (int64_t)1 << 30);
    gated_norm_kernel<T><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_norm(const NormParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
