// Selective scan with one decay per channel and state index:
//     s = delta + bias (through softplus),  h[n] = exp(s A[n]) h[n] + s u B[n]
//     y = (sum_n C[n] h[n] + D u) silu(z)
//
// With a decay of its own for every (channel, state index) the recurrence has
// no matrix-product form: it is N exponentials and 4 N fp32 operations per
// token and channel on the vector units, and that bounds a prompt (24 cycles
// of a SIMD per 64 states and token: 4 each for the product s A, the product
// s u B and the two accumulations, 8 for the exponential).  A single token is
// bounded by reading and writing the state.
//
// Prompt kernel.  A workgroup of four waves owns 64 channels of one sequence.
// In the scan, lane = channel and wave = a quarter of the states: h and A stay
// in N/4 registers each, B and C of a token are the same for all lanes (LDS
// broadcasts), and the four partial sums of y meet in LDS.  Everything that is
// per (token, channel) instead of per state - softplus, s u, the skip term, the
// gate, conversions and global accesses - is done once, tile by tile (32
// tokens), with 8 channels of one token per thread.  The next tile's global
// loads are in flight during a tile's scan.
//
// Few sequences and channels leave most of the GPU idle that way, and the
// recurrence is serial in tokens.  The tokens are then split into ranges: one
// launch runs every range but the last from a zero state (range 0 from
// init_state) without outputs and leaves its final state and the sum of its
// steps; in the second launch each range forms its entering state,
//     h <- exp(A sum_of_steps) h + range's final state,
// over the ranges before it, and runs in full.  That doubles the work, so
// ranges are used only where they at least quadruple the workgroups.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kChannels = 64;  // channels per workgroup: one per lane
constexpr int kWaves = 4;      // quarters of the states
constexpr int kTile = 32;      // tokens per tile
constexpr int kThreads = 64 * kWaves;
constexpr int kCh = 8;         // channels per thread in the per-(token, channel) work
static_assert(kTile * kChannels == kThreads * kCh, "one row piece per thread");

// 8 channels of one token as loaded: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Row8 {
    static constexpr int W = sizeof(T) * 8 / 16, VEC = 16 / sizeof(T);
    u32x4 v[W];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = load_words(p + k * VEC);
    }
    // Element by element, the last of `valid` repeated.
    __device__ __forceinline__ void load(const T *p, int valid) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int at = min(k * VEC, valid - 1);
            v[k] = load_first(p + at, valid - at);
        }
    }
    __device__ __forceinline__ float f32(int i) const { return word_f32(v[i / VEC], i % VEC, T()); }
};

// The accepted index of sequence b, clamped; seqlen where none is asked for.
__device__ __forceinline__ int64_t accepted(const SelectiveParams &p, int64_t b) {
    if (!p.state_out) return p.seqlen;
    const int64_t j = p.state_out_idx[b];
    return j < -1 ? -1 : (j > p.seqlen - 1 ? p.seqlen - 1 : j);
}

// STATES: leave the range's final state and sum of steps only.  ODD: a group's
// channels are no multiple of 8, so that rows are read element by element.
template <typename T, int N, bool STATES, bool ODD>
__global__ __launch_bounds__(kThreads) void scan_tiles_kernel(SelectiveParams p) {
    constexpr int NS = N / kWaves;        // states per lane
    constexpr int BCV = 2 * N / 4;        // 4-element pieces of a token's B and C
    constexpr int BCT = (kTile * BCV + kThreads - 1) / kThreads;
    __shared__ __align__(16) float dls[kTile][kChannels];
    __shared__ __align__(16) float dus[kTile][kChannels];
    __shared__ __align__(16) float bcs[kTile][2 * N];
    __shared__ __align__(16) float yps[STATES ? 1 : kWaves][STATES ? 1 : kTile][kChannels];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = (p.group_channels + kChannels - 1) / kChannels;
    const int ct = blockIdx.x % tiles, r = blockIdx.x / tiles;  // channel tile and token range
    const int g = blockIdx.y;
    const int64_t b = blockIdx.z;
    const int dg0 = ct * kChannels, d0 = g * p.group_channels + dg0;
    const int nch = min(kChannels, p.group_channels - dg0);
    const int64_t t_lo = (int64_t)r * p.range_len;
    const int64_t t_hi = min(t_lo + p.range_len, p.seqlen);

    // This thread's 8 channels of one token of a tile.
    const int row = tid >> 3, c8 = (tid & 7) * kCh;
    const int nv = max(0, min(kCh, nch - c8));
    // Where they are read: pieces past the tile's channels read its last
    // channels again, and nothing comes of them.
    const int from = d0 + (ODD ? min(c8, nch - 1) : min(c8, nch - kCh)), nread = ODD ? max(nv, 1) : kCh;
    const T *u = reinterpret_cast<const T *>(p.u) + b * p.u_bs + from;
    const T *dl = reinterpret_cast<const T *>(p.delta) + b * p.delta_bs + from;
    const T *z = !STATES && p.z ? reinterpret_cast<const T *>(p.z) + b * p.z_bs + from : nullptr;
    const T *B = reinterpret_cast<const T *>(p.B) + b * p.B_bs + g * N;
    const T *C = reinterpret_cast<const T *>(p.C) + b * p.C_bs + g * N;
    float bias[kCh], skip[kCh];
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
        bias[i] = p.delta_bias && i < nv ? p.delta_bias[d0 + c8 + i] : 0.0f;
        skip[i] = !STATES && p.D && i < nv ? p.D[d0 + c8 + i] : 0.0f;
    }

    // A tile's loads, none of them conditional so that they stay in flight.
    // Tokens past the range's end read its last row again (the scan stops
    // before them).
    Row8<T> ru, rd, rz;
    Pack<T, 4> rbc[BCT];
    auto load_tile = [&](int64_t t0) {
        const int64_t t = min(t0 + row, t_hi - 1);
        if constexpr (ODD) {
            ru.load(u + t * p.u_ts, nread);
            rd.load(dl + t * p.delta_ts, nread);
            if (z) rz.load(z + t * p.z_ts, nread);
        } else {
            ru.load(u + t * p.u_ts);
            rd.load(dl + t * p.delta_ts);
            if (z) rz.load(z + t * p.z_ts);
        }
#pragma unroll
        for (int k = 0; k < BCT; ++k) {
            const int e = min(tid + k * kThreads, kTile * BCV - 1), tr = e / BCV, c = (e - tr * BCV) * 4;
            const int64_t tb = min(t0 + tr, t_hi - 1);
            rbc[k] = *reinterpret_cast<const Pack<T, 4> *>(c < N ? B + tb * p.B_ts + c : C + tb * p.C_ts + c - N);
        }
    };
    load_tile(t_lo);

    // Entering state of this lane's channel and quarter of the states.
    const bool mine = lane < nch;
    const int64_t dn = (int64_t)(d0 + lane) * N + wave * NS;     // into [D,N]
    const int64_t at = b * p.channels * N + dn;                  // into [b,D,N]
    const int64_t slot = p.batch * p.channels * N;               // one range's states in the workspace
    float a[NS], h[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) a[n] = mine ? p.A[dn + n] * kLog2e : 0.0f;
    {
        // Range 0 of the full pass takes init_state from the first launch's
        // copy: the last range may be writing final_state over it by now.
        const float *first = !STATES && p.ranges > 1 ? p.range_state + (int64_t)(p.ranges - 1) * slot : p.init_state;
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = mine && p.init_state && r == 0 ? first[at + n] : 0.0f;
    }
    if (STATES) {
        if (r == 0 && p.init_state && mine)
#pragma unroll
            for (int n = 0; n < NS; ++n) p.range_state[(int64_t)(p.ranges - 1) * slot + at + n] = h[n];
    } else if (r > 0 && mine) {
#pragma unroll 4
        for (int k = 0; k < r; ++k) {
            const float sum = p.range_steps[((int64_t)k * p.batch + b) * p.channels + d0 + lane];
#pragma unroll
            for (int n = 0; n < NS; ++n)
                h[n] = fmaf(exp2_hw(sum * a[n]), h[n], p.range_state[(int64_t)k * slot + at + n]);
        }
    }
    const int64_t j = STATES ? p.seqlen : accepted(p, b);
    if (!STATES && p.state_out && j < 0 && r == 0 && mine)
#pragma unroll
        for (int n = 0; n < NS; ++n) p.state_out[at + n] = h[n];

    double steps = 0.0;  // sum of the range's steps, rounded once at the end
    T *y = STATES ? nullptr : reinterpret_cast<T *>(p.y) + (b * p.seqlen + row) * p.channels + d0 + c8;
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += kTile) {
        const int nt = (int)min((int64_t)kTile, t_hi - t0);
        // Per (token, channel): the step and s u; B and C to fp32.
        float uv[kCh];
        const Row8<T> zc = rz;
        {
            f32x4 dv[2], du[2];
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
                uv[i] = ru.f32(i);
                float s = rd.f32(i) + bias[i];
                if (p.softplus) s = softplus(s);
                dv[i >> 2][i & 3] = s;
                du[i >> 2][i & 3] = s * uv[i];
            }
            *reinterpret_cast<f32x4 *>(&dls[row][c8]) = dv[0];
            *reinterpret_cast<f32x4 *>(&dls[row][c8 + 4]) = dv[1];
            *reinterpret_cast<f32x4 *>(&dus[row][c8]) = du[0];
            *reinterpret_cast<f32x4 *>(&dus[row][c8 + 4]) = du[1];
#pragma unroll
            for (int k = 0; k < BCT; ++k) {
                const int e = tid + k * kThreads;
                if (e < kTile * BCV) {
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = to_f32(rbc[k].v[i]);
                    *reinterpret_cast<f32x4 *>(&bcs[e / BCV][(e % BCV) * 4]) = v;
                }
            }
        }
        if (t0 + kTile < t_hi) load_tile(t0 + kTile);
        lds_barrier();
        // The scan: tokens in order, split after the accepted index.
        auto token = [&](int t) {
            const float s = dls[t][lane], du = dus[t][lane];
            const float *bc = bcs[t] + wave * NS;
            float acc = 0.0f;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                h[n] = fmaf(exp2_hw(s * a[n]), h[n], du * bc[n]);
                if (!STATES) acc = n == 0 ? h[n] * bc[N] : fmaf(h[n], bc[N + n], acc);
            }
            if (STATES) {
                if (wave == 0) steps += (double)s;
            } else {
                yps[wave][t][lane] = acc;
            }
        };
        const bool here = !STATES && p.state_out && j >= t0 && j < t0 + nt;
        int t = 0;
        for (int part = 0; part < 2; ++part) {
            const int end = part == 0 && here ? (int)(j - t0) + 1 : nt;
            for (; t + 4 <= end; t += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) token(t + q);
            }
            for (; t < end; ++t) token(t);
            if (!here) break;
            if (part == 0 && mine)
#pragma unroll
                for (int n = 0; n < NS; ++n) p.state_out[at + n] = h[n];
        }
        lds_barrier();
        if (!STATES && row < nt && nv > 0) {
            // Per (token, channel): the four partial sums, skip, gate, store.
            Pack<T, kCh> o;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x4 v = *reinterpret_cast<const f32x4 *>(&yps[0][row][c8 + 4 * q]);
#pragma unroll
                for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4 *>(&yps[w][row][c8 + 4 * q]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 4 * q + i;
                    float f = fmaf(skip[c], uv[c], v[i]);
                    if (z) f *= silu(zc.f32(c));
                    o.v[c] = from_f32<T>(f);
                }
            }
            T *yr = y + t0 * p.channels;
            if constexpr (ODD) {
#pragma unroll
                for (int i = 0; i < kCh; ++i)
                    if (i < nv) yr[i] = o.v[i];
            } else {
                *reinterpret_cast<Pack<T, kCh> *>(yr) = o;
            }
        }
    }
    if (!mine) return;
    if (STATES) {
#pragma unroll
        for (int n = 0; n < NS; ++n) p.range_state[(int64_t)r * slot + at + n] = h[n];
        if (wave == 0) p.range_steps[((int64_t)r * p.batch + b) * p.channels + d0 + lane] = (float)steps;
    } else if (p.final_state && t_hi == p.seqlen) {
#pragma unroll
        for (int n = 0; n < NS; ++n) p.final_state[at + n] = h[n];
    }
}

// Sum over W = 2, 4, 8 or 16 adjacent lanes, in every one of them.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
    v += dpp<0xB1>(v);                         // quad_perm 1,0,3,2
    if constexpr (W >= 4) v += dpp<0x4E>(v);   // quad_perm 2,3,0,1
    if constexpr (W >= 8) v += dpp<0x141>(v);  // row_half_mirror: the other quad of 8 lanes
    if constexpr (W >= 16) v += dpp<0x140>(v); // row_mirror: the other 8 of 16 lanes
    return v;
}

// Few tokens: 4 states per lane, N/4 lanes per channel, so that the states are
// read and written in whole 16-byte pieces, each once.
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void scan_steps_kernel(SelectiveParams p) {
    constexpr int W = N / 4, CH = kThreads / W;
    const int tid = threadIdx.x, part = tid % W;
    const int dg = blockIdx.x * CH + tid / W;
    if (dg >= p.group_channels) return;  // whole groups of W lanes leave
    const int g = blockIdx.y, d = g * p.group_channels + dg;
    const int64_t b = blockIdx.z;
    const T *u = reinterpret_cast<const T *>(p.u) + b * p.u_bs + d;
    const T *dl = reinterpret_cast<const T *>(p.delta) + b * p.delta_bs + d;
    const T *z = p.z ? reinterpret_cast<const T *>(p.z) + b * p.z_bs + d : nullptr;
    const T *B = reinterpret_cast<const T *>(p.B) + b * p.B_bs + g * N + 4 * part;
    const T *C = reinterpret_cast<const T *>(p.C) + b * p.C_bs + g * N + 4 * part;
    T *y = reinterpret_cast<T *>(p.y) + b * p.seqlen * p.channels + d;
    const int64_t at = (b * p.channels + d) * N + 4 * part;
    f32x4 h = {0.f, 0.f, 0.f, 0.f}, a = h;
    if (p.init_state) h = *reinterpret_cast<const f32x4 *>(p.init_state + at);
    if (p.seqlen > 0) a = *reinterpret_cast<const f32x4 *>(p.A + (int64_t)d * N + 4 * part) * kLog2e;
    const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f, skip = p.D ? p.D[d] : 0.0f;
    const int64_t j = accepted(p, b);
    if (p.state_out && j < 0) *reinterpret_cast<f32x4 *>(p.state_out + at) = h;
    for (int64_t t = 0; t < p.seqlen; ++t) {
        const float uv = to_f32(u[t * p.u_ts]);
        float s = to_f32(dl[t * p.delta_ts]) + bias;
        const Pack<T, 4> bv = *reinterpret_cast<const Pack<T, 4> *>(B + t * p.B_ts);
        const Pack<T, 4> cv = *reinterpret_cast<const Pack<T, 4> *>(C + t * p.C_ts);
        const float zv = z ? to_f32(z[t * p.z_ts]) : 0.0f;
        if (p.softplus) s = softplus(s);
        const float du = s * uv;
        float acc = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            h[n] = fmaf(exp2_hw(s * a[n]), h[n], du * to_f32(bv.v[n]));
            acc = fmaf(h[n], to_f32(cv.v[n]), acc);
        }
        acc = fmaf(skip, uv, lanes_sum<W>(acc));
        if (z) acc *= silu(zv);
        if (part == 0) y[t * p.channels] = from_f32<T>(acc);
        if (p.state_out && t == j) *reinterpret_cast<f32x4 *>(p.state_out + at) = h;
    }
    if (p.final_state) *reinterpret_cast<f32x4 *>(p.final_state + at) = h;
}

// Calls up to this many tokens run without tiles.
constexpr int64_t kFewTokens = 16;

template <typename T, int N, bool ODD>
hipError_t run_tiles(const SelectiveParams &p, hipStream_t stream) {
    const unsigned tiles = (p.group_channels + kChannels - 1) / kChannels;
    if (p.ranges > 1) {
        const dim3 grid(tiles * (p.ranges - 1), p.ngroups, (unsigned)p.batch);
        scan_tiles_kernel<T, N, true, ODD><<<grid, kThreads, 0, stream>>>(p);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
    }
    const dim3 grid(tiles * p.ranges, p.ngroups, (unsigned)p.batch);
    scan_tiles_kernel<T, N, false, ODD><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t run(const SelectiveParams &p, hipStream_t stream) {
    if (p.seqlen <= kFewTokens) {
        constexpr int CH = kThreads / (N / 4);
        const dim3 grid((p.group_channels + CH - 1) / CH, p.ngroups, (unsigned)p.batch);
        scan_steps_kernel<T, N><<<grid, kThreads, 0, stream>>>(p);
        return hipGetLastError();
    }
    return p.group_channels % kCh == 0 ? run_tiles<T, N, false>(p, stream) : run_tiles<T, N, true>(p, stream);
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

void selective_ranges(SelectiveParams &p) {
    p.ranges = 1;
    p.range_len = (p.seqlen + kTile - 1) / kTile * kTile;
    if (p.seqlen <= kFewTokens || p.batch == 0) return;
    // Workgroups of an unsplit call; the GPU holds three per compute unit.
    const int64_t tiles = (p.group_channels + kChannels - 1) / kChannels;
    const int64_t wgs = tiles * p.ngroups * p.batch;
    constexpr int64_t kUnits = 256, kMinRange = 2 * kTile;
    const int64_t want = std::min((3 * kUnits) / wgs, (p.seqlen + kMinRange - 1) / kMinRange);
    if (want < 4) return;
    p.range_len = ((p.seqlen + want - 1) / want + kTile - 1) / kTile * kTile;
    p.ranges = (int)((p.seqlen + p.range_len - 1) / p.range_len);
}

hipError_t launch_selective_scan(const SelectiveParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? by_state<bf16>(p, stream) : by_state<float>(p, stream);
}

}  // namespace ssd
