// Selective scan with one decay per channel and state index:
//     s = delta + bias (through softplus),  h[n] = exp(s A[n]) h[n] + s u B[n]
//     y = (sum_n C[n] h[n] + D u) silu(z)
// A lane owns one channel with all its N states in registers and walks the
// tokens in order.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kLanes = 64;

template <typename T, int N>
__global__ __launch_bounds__(kLanes) void selective_scan_kernel(SelectiveParams p) {
    const int g = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int dg = blockIdx.x * kLanes + threadIdx.x;
    if (dg >= p.group_channels) return;
    const int d = g * p.group_channels + dg;
    const T *u = reinterpret_cast<const T *>(p.u) + b * p.u_bs + d;
    const T *dl = reinterpret_cast<const T *>(p.delta) + b * p.delta_bs + d;
    const T *z = p.z ? reinterpret_cast<const T *>(p.z) + b * p.z_bs + d : nullptr;
    const T *B = reinterpret_cast<const T *>(p.B) + b * p.B_bs + g * N;
    const T *C = reinterpret_cast<const T *>(p.C) + b * p.C_bs + g * N;
    T *y = reinterpret_cast<T *>(p.y) + b * p.seqlen * p.channels + d;
    const int64_t at = (b * p.channels + d) * N;

    float h[N], a[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        h[n] = p.init_state ? p.init_state[at + n] : 0.0f;
        a[n] = p.seqlen > 0 ? p.A[(int64_t)d * N + n] * kLog2e : 0.0f;
    }
    int64_t j = p.seqlen;  // no such token
    if (p.state_out) {
        j = p.state_out_idx[b];
        j = j < -1 ? -1 : (j > p.seqlen - 1 ? p.seqlen - 1 : j);
        if (j < 0)
            for (int n = 0; n < N; ++n) p.state_out[at + n] = h[n];
    }
    const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f, skip = p.D ? p.D[d] : 0.0f;
    for (int64_t t = 0; t < p.seqlen; ++t) {
        const float uv = to_f32(u[t * p.u_ts]);
        float s = to_f32(dl[t * p.delta_ts]) + bias;
        if (p.softplus) s = softplus(s);
        const float du = s * uv;
        float acc = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            h[n] = fmaf(exp2_hw(s * a[n]), h[n], du * to_f32(B[t * p.B_ts + n]));
            acc = fmaf(h[n], to_f32(C[t * p.C_ts + n]), acc);
        }
        acc = fmaf(skip, uv, acc);
        if (z) acc *= silu(to_f32(z[t * p.z_ts]));
        y[t * p.channels] = from_f32<T>(acc);
        if (t == j)
            for (int n = 0; n < N; ++n) p.state_out[at + n] = h[n];
    }
    if (p.final_state)
        for (int n = 0; n < N; ++n) p.final_state[at + n] = h[n];
}

template <typename T, int N>
hipError_t run(const SelectiveParams &p, hipStream_t stream) {
    const dim3 grid((p.group_channels + kLanes - 1) / kLanes, p.ngroups, (unsigned)p.batch);
    selective_scan_kernel<T, N><<<grid, kLanes, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t by_state(const SelectiveParams &p, hipStream_t stream) {
    switch (p.dstate) {
        case 8: return run<T, 8>(p, stream);
        case 16: return run<T, 16>(p, stream);
        case 32: return run<T, 32>(p, stream);
        default: return run<T, 64>(p, stream);
    }
}

}  // namespace

hipError_t launch_selective_scan(const SelectiveParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? by_state<bf16>(p, stream) : by_state<float>(p, stream);
}

}  // namespace ssd
