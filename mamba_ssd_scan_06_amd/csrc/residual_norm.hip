// Norms before and after a block with its gate, scales and the residual stream:
//
//     n   = x rsqrt(mean x^2 + eps) post_weight  (or x)
//     h   = residual_scale r + branch_scale layer_scale act(gate) n
//     out = h rsqrt(mean h^2 + eps) weight
//
// Up to three reads and two writes per element and nothing else: memory bound
// (16384 rows: 4096 channels of bf16 with everything 135 us, 5.0 TB/s; 5120 with an
// fp32 stream 179 us, 5.6 TB/s; one row 4 us, a launch).
// A row is held in the registers of `lanes` threads (a 16-byte piece of x each,
// up to four times, with the residual's and the gate's), so that both means are
// taken without reading anything twice; sums of squares are joined by shuffles
// and, beyond a wave, through LDS.  Rows beyond 1024 threads' registers are read
// once per mean and once more by a workgroup that loops over them.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kMaxHeld = 4;

struct RowGrid {
    int lanes;  // threads per row, a power of two; a workgroup has max(lanes, 64)
};

// Sum over a row's lanes (all of the workgroup where lanes > 64).  Calls take the
// two halves of `waves` in turn, so that the barrier of the one between stands
// between a half's reads and its next writes.
__device__ __forceinline__ float row_sum(float v, int lanes, float (&waves)[2][16], int &turn) {
    for (int m = 1; m < (lanes < 64 ? lanes : 64); m <<= 1) v += __shfl_xor(v, m);
    if (lanes > 64) {
        const int nw = lanes >> 6;
        float *sums = waves[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
        for (int w = 0; w < nw; ++w) v += sums[w];
    }
    return v;
}

// 1 / (1 + exp(-v)) for a result of type T; the same steps as silu's.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-v * kLog2e));
    const float e = exp_neg_abs(v);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float s = fmaf(fmaf(-r, e, 1.0f - r), r, r);
    return v < 0.0f ? e * s : s;
}

// VEC values of the residual stream, whose type may be wider than x's.
template <typename T, typename R>
struct StreamPiece {
    static constexpr int VEC = 16 / sizeof(T), WORDS = VEC * sizeof(R) / 16;
    u32x4 w[WORDS];
    __device__ __forceinline__ void load(const R *p) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = load_words(p + i * (VEC / WORDS));
    }
    __device__ __forceinline__ void load_part(const R *p, int valid) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            w[i] = i * (VEC / WORDS) < valid ? load_first(p + i * (VEC / WORDS), valid - i * (VEC / WORDS))
                                             : u32x4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ float get(int i) const { return word_f32(w[i / (VEC / WORDS)], i % (VEC / WORDS), R()); }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            float part[VEC / WORDS];
#pragma unroll
            for (int k = 0; k < VEC / WORDS; ++k) part[k] = v[i * (VEC / WORDS) + k];
            w[i] = to_words(part, R());
        }
    }
    __device__ __forceinline__ void store(R *p) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) store_words(p + i * (VEC / WORDS), w[i]);
    }
    __device__ __forceinline__ void store_part(R *p, int valid) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) store_first(p + i * (VEC / WORDS), w[i], valid - i * (VEC / WORDS));
    }
};

// VEC fp32 values of a vector over the channels.
template <int VEC>
struct Channels {
    u32x4 w[VEC / 4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = load_words(p + 4 * i);
    }
    __device__ __forceinline__ void load_part(const float *p, int valid) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            w[i] = 4 * i < valid ? load_first(p + 4 * i, valid - 4 * i) : u32x4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ float get(int i) const { return word_f32(w[i / 4], i % 4, float()); }
};

// HELD: pieces per thread; 0: any number (or a row shorter than a piece).  MAX:
// threads at most.  R: the residual stream's type, which also sets how exactly
// the gate's activation is computed.
template <typename T, typename R, int HELD, int MAX>
__global__ __launch_bounds__(MAX) void residual_norm_kernel(ResidualNormParams p, RowGrid gr) {
    constexpr int VEC = 16 / sizeof(T);
    typedef StreamPiece<T, R> Stream;
    __shared__ float waves[2][16];
    int turn = 0;
    const int lanes = gr.lanes, lane = threadIdx.x & (lanes - 1);
    const int per_wg = blockDim.x / lanes;
    // All threads of a workgroup take the same number of turns (barriers in
    // row_sum); those without a row of their own work on the last one and store
    // nothing.
    for (int64_t first = (int64_t)blockIdx.x * per_wg; first < p.rows; first += (int64_t)gridDim.x * per_wg) {
        const int64_t mine = first + threadIdx.x / lanes;
        const unsigned row = (unsigned)min(mine, p.rows - 1), b = row / (unsigned)p.seqlen,
                       t = row - b * (unsigned)p.seqlen;
        const T *x = reinterpret_cast<const T *>(p.x) + b * p.x_bs + t * p.x_ts;
        const R *res = p.residual ? reinterpret_cast<const R *>(p.residual) + b * p.r_bs + t * p.r_ts : nullptr;
        const T *gate = p.gate ? reinterpret_cast<const T *>(p.gate) + b * p.gate_bs + t * p.gate_ts : nullptr;
        T *out = reinterpret_cast<T *>(p.out) + (int64_t)row * p.dim;
        R *hout = p.residual_out ? reinterpret_cast<R *>(p.residual_out) + (int64_t)row * p.dim : nullptr;

        auto scale_of = [&](float sum) { return 1.0f / sqrtf(row_sum(sum, lanes, waves, turn) / (float)p.dim + p.eps); };
        // x -> h in place; n_scale is the first norm's factor (1 without it).
        auto stream_value = [&](float x_, float gate_, float post, float layer, float r_, float n_scale) {
            float v = x_ * n_scale;
            if (p.post_weight) v *= post;
            if (gate) v *= p.activation == 0 ? gate_ : p.activation == 1 ? silu<R>(gate_) : sigmoid<R>(gate_);
            if (p.layer_scale) v *= layer;
            v *= p.branch_scale;
            return res ? fmaf(p.residual_scale, r_, v) : v;
        };
        const u32x4 none = {0u, 0u, 0u, 0u};
        if constexpr (HELD > 0) {
            // A piece that would pass the row's end is moved back to end there.
            // The elements it then shares with the piece before it are left out
            // of the sums and stored twice with equal values (after every
            // lane's loads: the scale depends on them all).
            int at[HELD];
            u32x4 xr[HELD], gt[HELD];
            Stream rs[HELD];
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                at[m] = min((m * lanes + lane) * VEC, p.dim - VEC);
                xr[m] = load_words(x + at[m]);
                gt[m] = none;
                if (gate) gt[m] = load_words(gate + at[m]);
                if (res) rs[m].load(res + at[m]);
            }
            // Few rows wait for every load in turn, so the vectors over the
            // channels are loaded here too where a thread holds one piece.
            constexpr bool EARLY = HELD == 1;
            Channels<VEC> post = {}, layer = {}, w = {};
            if (EARLY && p.post_weight) post.load(p.post_weight + at[0]);
            if (EARLY && p.layer_scale) layer.load(p.layer_scale + at[0]);
            if (EARLY && p.weight) w.load(p.weight + at[0]);
            auto sum_of = [&](int m, const float (&v)[VEC], float sum) {
                const int shared = (m * lanes + lane) * VEC - at[m];  // all of them: no piece of its own
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = i >= shared ? fmaf(v[i], v[i], sum) : sum;
                return sum;
            };
            float n_scale = 1.0f;
            if (p.post_norm) {
                float sum = 0.0f;
#pragma unroll
                for (int m = 0; m < HELD; ++m) {
                    float v[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = word_f32(xr[m], i, T());
                    sum = sum_of(m, v, sum);
                }
                n_scale = scale_of(sum);
            }
            float v[HELD][VEC], sum = 0.0f;
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                if (!EARLY && p.post_weight) post.load(p.post_weight + at[m]);
                if (!EARLY && p.layer_scale) layer.load(p.layer_scale + at[m]);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[m][i] = stream_value(word_f32(xr[m], i, T()), word_f32(gt[m], i, T()), post.get(i), layer.get(i),
                                           res ? rs[m].get(i) : 0.0f, n_scale);
                sum = sum_of(m, v[m], sum);
            }
            const float scale = scale_of(sum);
#pragma unroll
            for (int m = 0; m < HELD; ++m) {
                if ((m * lanes + lane) * VEC - at[m] >= VEC || mine >= p.rows) continue;
                if (hout) {
                    Stream hs;
                    hs.set(v[m]);
                    hs.store(hout + at[m]);
                }
                if (!EARLY && p.weight) w.load(p.weight + at[m]);
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = p.weight ? v[m][i] * scale * w.get(i) : v[m][i] * scale;
                store_words(out + at[m], to_words(o, T()));
            }
        } else {
            // Whole pieces in a loop, the last, partial one by its lane.
            const int whole = p.dim / VEC * VEC, left = p.dim - whole;
            const bool last = left > 0 && (whole / VEC & (lanes - 1)) == lane;
            float n_scale = 1.0f;
            if (p.post_norm) {
                float sum = 0.0f;
                for (int c = lane * VEC; c < whole; c += lanes * VEC) {
                    const u32x4 xr = load_words(x + c);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum = fmaf(word_f32(xr, i, T()), word_f32(xr, i, T()), sum);
                }
                if (last) {
                    const u32x4 xr = load_first(x + whole, left);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        sum = i < left ? fmaf(word_f32(xr, i, T()), word_f32(xr, i, T()), sum) : sum;
                }
                n_scale = scale_of(sum);
            }
            auto piece = [&](int c, float (&v)[VEC]) {
                const u32x4 xr = load_words(x + c);
                u32x4 gt = none;
                if (gate) gt = load_words(gate + c);
                Stream rs;
                if (res) rs.load(res + c);
                Channels<VEC> post = {}, layer = {};
                if (p.post_weight) post.load(p.post_weight + c);
                if (p.layer_scale) layer.load(p.layer_scale + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[i] = stream_value(word_f32(xr, i, T()), word_f32(gt, i, T()), post.get(i), layer.get(i),
                                        res ? rs.get(i) : 0.0f, n_scale);
            };
            auto part = [&](float (&v)[VEC]) {
                const u32x4 xr = load_first(x + whole, left);
                u32x4 gt = none;
                if (gate) gt = load_first(gate + whole, left);
                Stream rs;
                if (res) rs.load_part(res + whole, left);
                Channels<VEC> post = {}, layer = {};
                if (p.post_weight) post.load_part(p.post_weight + whole, left);
                if (p.layer_scale) layer.load_part(p.layer_scale + whole, left);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[i] = stream_value(word_f32(xr, i, T()), word_f32(gt, i, T()), post.get(i), layer.get(i),
                                        res ? rs.get(i) : 0.0f, n_scale);
            };
            float v[VEC], sum = 0.0f;
            for (int c = lane * VEC; c < whole; c += lanes * VEC) {
                piece(c, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = fmaf(v[i], v[i], sum);
            }
            if (last) {
                part(v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum = i < left ? fmaf(v[i], v[i], sum) : sum;
            }
            const float scale = scale_of(sum);
            if (mine >= p.rows) continue;
            // Each lane stores the pieces that it reads itself, so that the
            // outputs may be x and the residual.
            for (int c = lane * VEC; c < whole; c += lanes * VEC) {
                piece(c, v);
                if (hout) {
                    Stream hs;
                    hs.set(v);
                    hs.store(hout + c);
                }
                Channels<VEC> w = {};
                if (p.weight) w.load(p.weight + c);
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = p.weight ? v[i] * scale * w.get(i) : v[i] * scale;
                store_words(out + c, to_words(o, T()));
            }
            if (last) {
                part(v);
                if (hout) {
                    Stream hs;
                    hs.set(v);
                    hs.store_part(hout + whole, left);
                }
                Channels<VEC> w = {};
                if (p.weight) w.load_part(p.weight + whole, left);
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = p.weight ? v[i] * scale * w.get(i) : v[i] * scale;
                store_first(out + whole, to_words(o, T()), left);
            }
        }
    }
}

template <typename T, typename R, int HELD>
hipError_t launch(const ResidualNormParams &p, const RowGrid &gr, unsigned grid, int threads, hipStream_t stream) {
    if constexpr (HELD < kMaxHeld)  // four pieces: 1024 lanes only
        if (threads <= 256) {
            residual_norm_kernel<T, R, HELD, 256><<<grid, threads, 0, stream>>>(p, gr);
            return hipGetLastError();
        }
    residual_norm_kernel<T, R, HELD, 1024><<<grid, threads, 0, stream>>>(p, gr);
    return hipGetLastError();
}

template <typename T, typename R>
hipError_t run(const ResidualNormParams &p, hipStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    const int pieces = (p.dim + VEC - 1) / VEC;
    // The fewest lanes (at least 8) with three pieces each or fewer, and more while
    // that leaves less than eight waves per compute unit (256 rows of 4096 7.4 us with
    // less than four, 6.2 with eight; sixteen splits 300 fp32 rows of 5120 once more:
    // 8.7 and 12 us).  Four pieces leave too few
    // waves for the loads: 16384 rows of 4096 with everything 150 us with four, 136
    // with two of twice the lanes; three in the place of two of twice the lanes, of
    // which the last are partly idle: rows of 5120 179 and 205 us.
    RowGrid gr = {8};
    while (gr.lanes < 1024 && (pieces + gr.lanes - 1) / gr.lanes > 3) gr.lanes *= 2;
    while (gr.lanes < 1024 && pieces > gr.lanes && p.rows * gr.lanes < 8 * 256 * 64) gr.lanes *= 2;
    const int each = (pieces + gr.lanes - 1) / gr.lanes;
    const int held = p.dim < VEC || each > kMaxHeld ? 0 : each;
    const int threads = std::max(gr.lanes, 64);
    const int64_t wgs = (p.rows * gr.lanes + threads - 1) / threads;
    // A launch's threads stay below 2^32: 2^31 at most with 1024 per workgroup
    // (the workgroups take turns where there are more rows).
    const unsigned grid = (unsigned)std::min<int64_t>(wgs, (int64_t)1 << 21);
    switch (held) {
        case 1: return launch<T, R, 1>(p, gr, grid, threads, stream);
        case 2: return launch<T, R, 2>(p, gr, grid, threads, stream);
        case 3: return launch<T, R, 3>(p, gr, grid, threads, stream);
        case 4: return launch<T, R, 4>(p, gr, grid, threads, stream);
        default: return launch<T, R, 0>(p, gr, grid, threads, stream);
    }
}

}  // namespace

hipError_t launch_residual_norm(const ResidualNormParams &p, Elem e, Elem stream_elem, hipStream_t stream) {
    if (e == Elem::F32) return run<float, float>(p, stream);
    return stream_elem == Elem::F32 ? run<bf16, float>(p, stream) : run<bf16, bf16>(p, stream);
}

}  // namespace ssd
