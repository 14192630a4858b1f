// RMS norm with a gate over each of a row's ngroups parts:
//     v = x silu(z), out = v rsqrt(mean v^2 + eps) weight      (gate first), or
//     out = x rsqrt(mean x^2 + eps) weight silu(z)             (norm first).
//
// Two reads and one write per element: memory bound.  A part is held in the
// registers of `lanes` threads (16 bytes of x and z each, up to five times),
// so both inputs are read once; the sum of squares is joined by shuffles and,
// beyond a wave, through LDS.  Parts beyond 1024 threads' registers are read
// twice, by a workgroup that loops over them.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kMaxHeld = 5;  // 16-byte pieces a thread may hold

// Lanes: threads per part, a power of two; blockDim.x is max(lanes, 256) or lanes.
struct NormGrid {
    int lanes;
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_piece(const T *p, int valid) {
    if (valid >= VEC) return *reinterpret_cast<const Pack<T, VEC> *>(p);
    Pack<T, VEC> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = i < valid ? p[i] : from_f32<T>(0.0f);
    return r;
}

// Sum over a part's lanes (all of the workgroup where lanes > 64).
__device__ __forceinline__ float part_sum(float v, int lanes, float *waves) {
    for (int m = 1; m < (lanes < 64 ? lanes : 64); m <<= 1) v += __shfl_xor(v, m);
    if (lanes > 64) {
        const int nw = lanes >> 6;
        if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
        for (int w = 0; w < nw; ++w) v += waves[w];
        __syncthreads();  // the next part may write waves again
    }
    return v;
}

// HELD: pieces per thread; 0: any number, read twice.  MAX: threads at most.
template <typename T, int HELD, int MAX>
__global__ __launch_bounds__(MAX) void gated_norm_kernel(NormParams p, NormGrid gr) {
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float waves[16];
    const int lanes = gr.lanes, lane = threadIdx.x & (lanes - 1);
    const int per_wg = blockDim.x / lanes;
    const int64_t parts = p.rows * p.ngroups;
    // All threads of a workgroup take the same number of turns (barriers in
    // part_sum); those without a part of their own work on the last one and
    // store nothing.
    for (int64_t first = (int64_t)blockIdx.x * per_wg; first < parts; first += (int64_t)gridDim.x * per_wg) {
        const int64_t mine = first + threadIdx.x / lanes, k = min(mine, parts - 1);
        const unsigned row = (unsigned)(k / p.ngroups), b = row / (unsigned)p.seqlen, t = row - b * (unsigned)p.seqlen;
        const int c0 = (int)(k - (int64_t)row * p.ngroups) * p.group_dim;
        const T *x = reinterpret_cast<const T *>(p.x) + b * p.x_bs + t * p.x_ts + c0;
        const T *z = p.z ? reinterpret_cast<const T *>(p.z) + b * p.z_bs + t * p.z_ts + c0 : nullptr;
        T *out = reinterpret_cast<T *>(p.out) + (int64_t)row * p.dim + c0;
        const float *weight = p.weight ? p.weight + c0 : nullptr;

        auto finish = [&](const float (&v)[VEC], const Pack<T, VEC> &zr, float scale, int c) {
            const int valid = p.group_dim - c;
            const Pack<float, VEC> wv = weight ? load_piece<float, VEC>(weight + c, valid) : Pack<float, VEC>{};
            Pack<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float f = v[i] * scale;
                if (weight) f *= wv.v[i];
                if (z && p.norm_before_gate) f *= silu(to_f32(zr.v[i]));
                o.v[i] = from_f32<T>(f);
            }
            if (mine >= parts) return;
            if (valid >= VEC) {
                *reinterpret_cast<Pack<T, VEC> *>(out + c) = o;
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (i < valid) out[c + i] = o.v[i];
            }
        };
        // The values to normalise; they include the gate where it comes first.
        auto values = [&](const Pack<T, VEC> &xr, const Pack<T, VEC> &zr, float (&v)[VEC]) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[i] = to_f32(xr.v[i]);
                if (z && !p.norm_before_gate) v[i] *= silu(to_f32(zr.v[i]));
            }
        };
        if constexpr (HELD > 0) {
            Pack<T, VEC> xr[HELD], zr[HELD];
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                const int c = (m * lanes + lane) * VEC;
                xr[m] = load_piece<T, VEC>(x + c, max(p.group_dim - c, 0));
                if (z) zr[m] = load_piece<T, VEC>(z + c, max(p.group_dim - c, 0));
            }
            float v[HELD][VEC], sum = 0.0f;
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                values(xr[m], zr[m], v[m]);
                const int left = p.group_dim - (m * lanes + lane) * VEC;  // elements past the part's end count as 0
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = i < left ? fmaf(v[m][i], v[m][i], sum) : sum;
            }
            const float scale = 1.0f / sqrtf(part_sum(sum, lanes, waves) / (float)p.group_dim + p.eps);
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                const int c = (m * lanes + lane) * VEC;
                if (c < p.group_dim) finish(v[m], zr[m], scale, c);
            }
        } else {
            float v[VEC], sum = 0.0f;
            auto piece = [&](int c) {
                Pack<T, VEC> zr = {};
                if (z) zr = load_piece<T, VEC>(z + c, p.group_dim - c);
                values(load_piece<T, VEC>(x + c, p.group_dim - c), zr, v);
                return zr;
            };
            for (int c = lane * VEC; c < p.group_dim; c += lanes * VEC) {
                piece(c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = c + i < p.group_dim ? fmaf(v[i], v[i], sum) : sum;
            }
            const float scale = 1.0f / sqrtf(part_sum(sum, lanes, waves) / (float)p.group_dim + p.eps);
            for (int c = lane * VEC; c < p.group_dim; c += lanes * VEC) {
                const Pack<T, VEC> zr = piece(c);
                finish(v, zr, scale, c);
            }
        }
    }
}

template <typename T, int HELD>
hipError_t launch(const NormParams &p, const NormGrid &gr, unsigned grid, int threads, hipStream_t stream) {
    if (threads <= 256)
        gated_norm_kernel<T, HELD, 256><<<grid, threads, 0, stream>>>(p, gr);
    else
        gated_norm_kernel<T, HELD, 1024><<<grid, threads, 0, stream>>>(p, gr);
    return hipGetLastError();
}

template <typename T>
hipError_t run(const NormParams &p, hipStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    const int pieces = (p.group_dim + VEC - 1) / VEC;
    // The fewest lanes whose registers hold a part; at least 8.
    NormGrid gr = {8};
    while (gr.lanes < 1024 && (pieces + gr.lanes - 1) / gr.lanes > kMaxHeld) gr.lanes *= 2;
    const int held = (pieces + gr.lanes - 1) / gr.lanes;
    const int threads = std::max(gr.lanes, 64);
    const int64_t parts = p.rows * p.ngroups;
    const int64_t wgs = (parts * gr.lanes + threads - 1) / threads;
    const unsigned grid = (unsigned)std::min<int64_t>(wgs, (int64_t)1 << 22);
    switch (held) {
        case 1: return launch<T, 1>(p, gr, grid, threads, stream);
        case 2: return launch<T, 2>(p, gr, grid, threads, stream);
        case 3: return launch<T, 3>(p, gr, grid, threads, stream);
        case 4: return launch<T, 4>(p, gr, grid, threads, stream);
        case 5: return launch<T, 5>(p, gr, grid, threads, stream);
        default: return launch<T, 0>(p, gr, grid, threads, stream);
    }
}

}  // namespace

hipError_t launch_gated_norm(const NormParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
