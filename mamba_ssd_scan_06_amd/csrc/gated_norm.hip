// RMS norm with a gate over each of a row's ngroups parts:
//     v = x silu(z), out = v rsqrt(mean v^2 + eps) weight      (gate first), or
//     out = x rsqrt(mean x^2 + eps) weight silu(z)             (norm first).
//
// Two reads and one write per element: memory bound.  A part is held in the
// registers of `lanes` threads (16 bytes of x and z each, up to five times),
// so both inputs are read once; the sum of squares is joined by shuffles and,
// beyond a wave, through LDS (16384 rows of 5120 bf16: 98-104 us, 5 TB/s).
// Parts beyond 1024 threads' registers are read twice, by a workgroup that
// loops over them.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kMaxHeld = 5;  // 16-byte pieces a thread may hold

struct NormGrid {
    int lanes;  // threads per part, a power of two; a workgroup has max(lanes, 64)
};

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

// HELD: pieces per thread; 0: any number (or a part shorter than a piece),
// read twice.  MAX: threads at most.
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

        // The values to normalise; they include the gate where it comes first.
        auto values = [&](const u32x4 &xr, const u32x4 &zr, float (&v)[VEC]) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[i] = word_f32(xr, i, T());
                if (z && !p.norm_before_gate) v[i] *= silu<T>(word_f32(zr, i, T()));
            }
        };
        auto scaled = [&](const float (&v)[VEC], const u32x4 &zr, const u32x4 (&wv)[VEC / 4], float scale) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float f = v[i] * scale;
                if (weight) f *= word_f32(wv[i / 4], i % 4, float());
                if (z && p.norm_before_gate) f *= silu<T>(word_f32(zr, i, T()));
                o[i] = f;
            }
            return to_words(o, T());
        };
        auto scale_of = [&](float sum) { return 1.0f / sqrtf(part_sum(sum, lanes, waves) / (float)p.group_dim + p.eps); };
        const u32x4 none = {0u, 0u, 0u, 0u};
        if constexpr (HELD > 0) {
            // A piece that would pass the part's end is moved back to end
            // there.  The elements it then shares with the piece before it
            // are left out of the sum and stored twice with equal values
            // (after every lane's loads: the scale depends on them all).
            int at[HELD];
            u32x4 xr[HELD], zr[HELD];
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                at[m] = min((m * lanes + lane) * VEC, p.group_dim - VEC);
                xr[m] = load_words(x + at[m]);
                zr[m] = z ? load_words(z + at[m]) : none;
            }
            float v[HELD][VEC], sum = 0.0f;
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                values(xr[m], zr[m], v[m]);
                const int shared = (m * lanes + lane) * VEC - at[m];  // all of them: no piece of its own
                if (shared == 0) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum = fmaf(v[m][i], v[m][i], sum);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum = i >= shared ? fmaf(v[m][i], v[m][i], sum) : sum;
                }
            }
            const float scale = scale_of(sum);
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                if ((m * lanes + lane) * VEC - at[m] >= VEC || mine >= parts) continue;
                u32x4 wv[VEC / 4] = {};
                if (weight)
#pragma unroll
                    for (int i = 0; i < VEC / 4; ++i) wv[i] = load_words(weight + at[m] + 4 * i);
                store_words(out + at[m], scaled(v[m], zr[m], wv, scale));
            }
        } else {
            // Whole pieces in a loop, the last, partial one by its lane.
            const int whole = p.group_dim / VEC * VEC, left = p.group_dim - whole;
            const bool last = left > 0 && (whole / VEC & (lanes - 1)) == lane;
            float v[VEC], sum = 0.0f;
            for (int c = lane * VEC; c < whole; c += lanes * VEC) {
                values(load_words(x + c), z ? load_words(z + c) : none, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = fmaf(v[i], v[i], sum);
            }
            if (last) {
                values(load_first(x + whole, left), z ? load_first(z + whole, left) : none, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = i < left ? fmaf(v[i], v[i], sum) : sum;
            }
            const float scale = scale_of(sum);
            if (mine >= parts) continue;
            for (int c = lane * VEC; c < whole; c += lanes * VEC) {
                const u32x4 zr = z ? load_words(z + c) : none;
                values(load_words(x + c), zr, v);
                u32x4 wv[VEC / 4] = {};
                if (weight)
#pragma unroll
                    for (int i = 0; i < VEC / 4; ++i) wv[i] = load_words(weight + c + 4 * i);
                store_words(out + c, scaled(v, zr, wv, scale));
            }
            if (last) {
                const u32x4 zr = z ? load_first(z + whole, left) : none;
                values(load_first(x + whole, left), zr, v);
                u32x4 wv[VEC / 4] = {};
                if (weight)
#pragma unroll
                    for (int i = 0; i < VEC / 4; ++i)
                        if (4 * i < left) wv[i] = load_first(weight + whole + 4 * i, left - 4 * i);
                store_first(out + whole, scaled(v, zr, wv, scale), left);
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
    // The fewest lanes whose registers hold a part (at least 8), and more
    // while that leaves less than four waves per compute unit.
    const int64_t parts = p.rows * p.ngroups;
    NormGrid gr = {8};
    while (gr.lanes < 1024 && (pieces + gr.lanes - 1) / gr.lanes > kMaxHeld) gr.lanes *= 2;
    while (gr.lanes < 1024 && pieces > gr.lanes && parts * gr.lanes < 4 * 256 * 64) gr.lanes *= 2;
    const int held = p.group_dim < VEC ? 0 : (pieces + gr.lanes - 1) / gr.lanes;
    const int threads = std::max(gr.lanes, 64);
    const int64_t wgs = (parts * gr.lanes + threads - 1) / threads;
    // A launch's threads stay below 2^32: 2^31 at most with 1024 per workgroup
    // (the workgroups take turns where there are more parts).
    const unsigned grid = (unsigned)std::min<int64_t>(wgs, (int64_t)1 << 21);
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
