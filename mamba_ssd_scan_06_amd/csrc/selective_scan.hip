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
// loads are in flight during a tile's scan.  Measured: 394 us for 8 x 2048
// tokens of 5120 channels (N 16; up to 500 in the first sixty calls after an
// idle time), 31 VALU instructions per wave and token, 20 of them the scan's;
// the VALU is 92% busy where a compute unit holds three workgroups.  (Reading
// the next tokens' LDS values ahead into registers was slower: 445-490 us
// against 400-410.)
//
// Few sequences and channels leave most of the GPU idle that way, and the
// recurrence is serial in tokens.  The tokens are then split into ranges: one
// launch runs every range but the last from a zero state (range 0 from
// init_state) without outputs and leaves its final state and the sum of its
// steps; in the second launch each range forms its entering state,
//     h <- exp(A sum_of_steps) h + range's final state,
// over the ranges before it (scaled_by_exp2 where A or the steps let that
// factor grow), and runs in full.  That doubles the work, so ranges are used
// only where the GPU has room for four times the workgroups (selective_ranges
// has the figures).
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
    // 16 bytes from each of the offsets.
    __device__ __forceinline__ void load(const T *p, const int (&at)[W]) {
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = load_words(p + at[k]);
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

// h 2^x for any x: the power's whole part goes into h's exponent, so that it
// overflows or vanishes only where the product does (0 stays 0; beyond 2^300
// either way nothing of fp32 is left).
__device__ __forceinline__ float scaled_by_exp2(float h, float x) {
    x = fminf(fmaxf(x, -300.0f), 300.0f);
    const float whole = ceilf(x);
    return ldexpf(h * exp2_hw(x - whole), (int)whole);
}

// STATES: leave the range's final state and sum of steps only.  ODD: a group's
// channels are no multiple of 16 bytes, so that rows are read element by element.
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
    // Where they are read, in vectors of 16 bytes: those past the tile's
    // channels read its last ones again, and nothing comes of them.
    constexpr int VEC = Row8<T>::VEC, VECS = Row8<T>::W;
    int off[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k) off[k] = ODD ? min(c8, nch - 1) : min(c8 + k * VEC, nch - VEC);
    const int nread = max(nv, 1);  // ODD: elements from off[0] on
    const T *u = reinterpret_cast<const T *>(p.u) + b * p.u_bs + d0;
    const T *dl = reinterpret_cast<const T *>(p.delta) + b * p.delta_bs + d0;
    const bool gated = !STATES && p.z != nullptr;
    const T *z = reinterpret_cast<const T *>(p.z) + (gated ? b * p.z_bs + d0 : 0);
    const T *B = reinterpret_cast<const T *>(p.B) + b * p.B_bs + g * N;
    const T *C = reinterpret_cast<const T *>(p.C) + b * p.C_bs + g * N;
    float bias[kCh], skip[kCh];
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
        const int c = d0 + (ODD ? off[0] + min(i, nread - 1) : off[i / VEC] + i % VEC);
        bias[i] = p.delta_bias ? p.delta_bias[c] : 0.0f;
        skip[i] = !STATES && p.D ? p.D[c] : 0.0f;
    }

    // A tile's loads, none of them conditional so that they stay in flight.
    // Tokens past the range's end read its last row again (the scan stops
    // before them).
    Row8<T> ru, rd, rz;
    Pack<T, 4> rbc[BCT];
    auto load_tile = [&](int64_t t0) {
        const int left = (int)min(t_hi - t0, (int64_t)kTile) - 1;  // last token of the tile
        const int tr = min(row, left);
        const T *pu = u + t0 * p.u_ts + tr * p.u_ts, *pd = dl + t0 * p.delta_ts + tr * p.delta_ts,
                *pz = z + t0 * p.z_ts + tr * p.z_ts;
        if constexpr (ODD) {
            ru.load(pu + off[0], nread);
            rd.load(pd + off[0], nread);
            if (gated) rz.load(pz + off[0], nread);
        } else {
            ru.load(pu, off);
            rd.load(pd, off);
            if (gated) rz.load(pz, off);
        }
        const T *Bt = B + t0 * p.B_ts, *Ct = C + t0 * p.C_ts;
#pragma unroll
        for (int k = 0; k < BCT; ++k) {
            const int e = min(tid + k * kThreads, kTile * BCV - 1), c = e % BCV * 4;
            const int tb = min(e / BCV, left);
            rbc[k] = *reinterpret_cast<const Pack<T, 4> *>(c < N ? Bt + tb * p.B_ts + c : Ct + tb * p.C_ts + c - N);
        }
    };
    load_tile(t_lo);

    // Entering state of this lane's channel and quarter of the states.  Lanes
    // past the tile's channels carry its last one along and store nothing.
    const bool mine = lane < nch;
    const int d = d0 + min(lane, nch - 1);
    const int64_t dn = (int64_t)d * N + wave * NS;               // into [D,N]
    const int64_t at = b * p.channels * N + dn;                  // into [b,D,N]
    const int64_t slot = p.batch * p.channels * N;               // one range's states in the workspace
    float a[NS], h[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) a[n] = p.A[dn + n] * kLog2e;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = 0.0f;
    if (p.init_state && r == 0) {
        // Range 0 of the full pass takes init_state from the first launch's
        // copy: the last range may be writing final_state over it by now.
        const float *first = !STATES && p.ranges > 1 ? p.range_state + (int64_t)(p.ranges - 1) * slot : p.init_state;
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = first[at + n];
        if (STATES && mine)
#pragma unroll
            for (int n = 0; n < NS; ++n) p.range_state[(int64_t)(p.ranges - 1) * slot + at + n] = h[n];
    }
    if (!STATES && r > 0) {
        constexpr int U = NS > 8 ? 4 : 8;  // ranges whose loads are in flight together
        const float *st = p.range_state + at, *su = p.range_steps + b * p.channels + d;
        float a_most = a[0];
#pragma unroll
        for (int n = 1; n < NS; ++n) a_most = fmaxf(a_most, a[n]);
        for (int k0 = 0; k0 < r; k0 += U) {
            float sum[U], hr[U][NS];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int k = min(k0 + q, r - 1);
                sum[q] = su[(int64_t)k * p.batch * p.channels];
#pragma unroll
                for (int n = 0; n < NS; ++n) hr[q][n] = st[(int64_t)k * slot + n];
            }
            float sum_least = sum[0];
#pragma unroll
            for (int q = 1; q < U; ++q) sum_least = fminf(sum_least, sum[q]);
            // A decay that may grow (A > 0, or steps < 0) takes another way,
            // chosen by the wave: its factor over a whole range may pass the
            // fp32 range where the state does not, and an empty state's 0
            // times +inf would be NaN.
            if (__builtin_expect(__any(a_most > 0.0f || sum_least < 0.0f), 0)) {
#pragma unroll
                for (int q = 0; q < U; ++q)
                    if (k0 + q < r)
#pragma unroll
                        for (int n = 0; n < NS; ++n) h[n] = scaled_by_exp2(h[n], sum[q] * a[n]) + hr[q][n];
            } else {
#pragma unroll
                for (int q = 0; q < U; ++q)
                    if (k0 + q < r)
#pragma unroll
                        for (int n = 0; n < NS; ++n) h[n] = fmaf(exp2_hw(sum[q] * a[n]), h[n], hr[q][n]);
            }
        }
    }
    const int64_t j = STATES ? p.seqlen : accepted(p, b);
    if (!STATES && p.state_out && j < 0 && r == 0 && mine)
#pragma unroll
        for (int n = 0; n < NS; ++n) p.state_out[at + n] = h[n];

    // h and a have arrived: without this the compiler waits for every load in
    // flight where the scan first uses them, in each tile.
    wait_vmcnt<0>();
    double steps = 0.0;  // sum of the range's steps (this wave's part), rounded once at the end
    T *y = STATES ? nullptr : reinterpret_cast<T *>(p.y) + (b * p.seqlen + row) * p.channels + d0 + c8;
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += kTile) {
        const int nt = (int)min((int64_t)kTile, t_hi - t0);
        // Per (token, channel): the step and s u; B and C to fp32.
        float uv[kCh];
        const Row8<T> zc = rz;
        {
            f32x4 dv[2], du[2];
#pragma unroll
            for (int i = 0; i < kCh; ++i) dv[i >> 2][i & 3] = rd.f32(i) + bias[i];
            if (p.softplus) {
#pragma unroll
                for (int i = 0; i < kCh; ++i) dv[i >> 2][i & 3] = softplus(dv[i >> 2][i & 3]);
            }
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
                uv[i] = ru.f32(i);
                du[i >> 2][i & 3] = dv[i >> 2][i & 3] * uv[i];
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
            if (!STATES) yps[wave][t][lane] = acc;
        };
        const bool here = !STATES && p.state_out && j >= t0 && j < t0 + nt;
        int t = 0;
        for (int part = 0; part < 2; ++part) {
            const int end = part == 0 && here ? (int)(j - t0) + 1 : nt;
            // Tokens per turn: with 16 states per lane four would hold the
            // registers of two workgroups (8 x 1000 tokens of 2048 channels,
            // N 64: 336 us; two: 288; one: 331).
            constexpr int UN = NS >= 8 ? 2 : 4;
            for (; t + UN <= end; t += UN) {
#pragma unroll
                for (int q = 0; q < UN; ++q) token(t + q);
            }
            for (; t < end; ++t) token(t);
            if (!here) break;
            if (part == 0 && mine)
#pragma unroll
                for (int n = 0; n < NS; ++n) p.state_out[at + n] = h[n];
        }
        if (STATES) {
            // The sum of steps, a quarter of the tokens per wave.
            constexpr int PART = kTile / kWaves;
#pragma unroll
            for (int k = 0; k < PART; ++k)
                if (wave * PART + k < nt) steps += (double)dls[wave * PART + k][lane];
        }
        lds_barrier();
        if (!STATES && row < nt && nv > 0) {
            // Per (token, channel): the four partial sums, skip, gate, store.
            float f[kCh];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x4 v = *reinterpret_cast<const f32x4 *>(&yps[0][row][c8 + 4 * q]);
#pragma unroll
                for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4 *>(&yps[w][row][c8 + 4 * q]);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[4 * q + i] = fmaf(skip[4 * q + i], uv[4 * q + i], v[i]);
            }
            if (gated) {
#pragma unroll
                for (int i = 0; i < kCh; ++i) f[i] *= silu<T>(zc.f32(i));
            }
            T *yr = y + t0 * p.channels;
            if constexpr (ODD) {
#pragma unroll
                for (int i = 0; i < kCh; ++i)
                    if (i < nv) yr[i] = from_f32<T>(f[i]);
            } else {
#pragma unroll
                for (int k = 0; k < VECS; ++k) {
                    float part[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) part[i] = f[k * VEC + i];
                    if (k * VEC < nv) store_words(yr + k * VEC, to_words(part, T()));
                }
            }
        }
    }
    if (STATES) {
        // The waves' parts meet in LDS (its last readers are past a barrier).
        double *parts = reinterpret_cast<double *>(&dls[0][0]);
        parts[wave * 64 + lane] = steps;
        lds_barrier();
        if (wave == 0 && mine) {
            for (int w = 1; w < kWaves; ++w) steps += parts[w * 64 + lane];
            p.range_steps[((int64_t)r * p.batch + b) * p.channels + d] = (float)steps;
        }
    }
    if (!mine) return;
    if (STATES) {
#pragma unroll
        for (int n = 0; n < NS; ++n) p.range_state[(int64_t)r * slot + at + n] = h[n];
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

// Lane k of each quad, in all four of its lanes.
template <int K>
__device__ __forceinline__ float of_quad(float v) {
    return dpp<K * 0x55>(v);
}
// v[k] summed over W = 4, 8 or 16 adjacent lanes, in the lanes at place k of
// each quad.
template <int W>
__device__ __forceinline__ float lanes_sum4(const float (&v)[4]) {
    const int q = threadIdx.x & 3;
    // Halves, then quarters: each step keeps the values the lane's place asks
    // for and hands the others over.
    const float keep0 = q & 2 ? v[2] : v[0], give0 = q & 2 ? v[0] : v[2];
    const float keep1 = q & 2 ? v[3] : v[1], give1 = q & 2 ? v[1] : v[3];
    const float a = keep0 + dpp<0x4E>(give0), b = keep1 + dpp<0x4E>(give1);
    float r = (q & 1 ? b : a) + dpp<0xB1>(q & 1 ? a : b);
    if constexpr (W == 8) r += dpp<0x141>(dpp<0x1B>(r));  // the other quad: each reversed, then both mirrored
    if constexpr (W == 16) {
        r += dpp<0x124>(r);  // row_ror 4, then 8: all four quads of the row
        r += dpp<0x128>(r);
    }
    return r;
}

// Few tokens: 4 states per lane, N/4 lanes per channel, so that the states are
// read and written in whole 16-byte pieces, each once.  Four tokens go
// together where there are as many (and the accepted index is not among
// them): each lane of a quad does one token's softplus, gate and store, which
// are the same for all states.
template <typename T, int N, bool ONE>
__global__ __launch_bounds__(kThreads) void scan_steps_kernel(SelectiveParams p) {
    constexpr int W = N / 4, CH = kThreads / W;
    const int tid = threadIdx.x, part = tid % W;
    const int dg = blockIdx.x * CH + tid / W;
    if (dg >= p.group_channels) return;  // whole groups of W lanes leave
    const int g = blockIdx.y, d = g * p.group_channels + dg;
    const int64_t b = blockIdx.z;
    const int len = (int)p.seqlen;
    // Token rows as uniform pointers plus a lane's own offset in them.
    const T *u = reinterpret_cast<const T *>(p.u) + b * p.u_bs;
    const T *dl = reinterpret_cast<const T *>(p.delta) + b * p.delta_bs;
    const T *z = reinterpret_cast<const T *>(p.z) + (p.z ? b * p.z_bs : 0);
    const T *B = reinterpret_cast<const T *>(p.B) + b * p.B_bs + g * N;
    const T *C = reinterpret_cast<const T *>(p.C) + b * p.C_bs + g * N;
    T *y = reinterpret_cast<T *>(p.y) + b * p.seqlen * p.channels;
    const int64_t at = (b * p.channels + d) * N + 4 * part;
    f32x4 h = {0.f, 0.f, 0.f, 0.f}, a = h;
    if (p.init_state) h = *reinterpret_cast<const f32x4 *>(p.init_state + at);
    if (len > 0) a = *reinterpret_cast<const f32x4 *>(p.A + (int64_t)d * N + 4 * part) * kLog2e;
    const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f, skip = p.D ? p.D[d] : 0.0f;
    const int j = (int)accepted(p, b);
    if (p.state_out && j < 0) *reinterpret_cast<f32x4 *>(p.state_out + at) = h;

    auto advance = [&](float s, float du, const Pack<T, 4> &bv, const Pack<T, 4> &cv) {
        float acc = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            h[n] = fmaf(exp2_hw(s * a[n]), h[n], du * to_f32(bv.v[n]));
            acc = fmaf(h[n], to_f32(cv.v[n]), acc);
        }
        return acc;
    };
    auto piece = [&](const T *row) { return *reinterpret_cast<const Pack<T, 4> *>(row + 4 * part); };
    auto one = [&](int64_t t) {
        const float uv = to_f32((u + t * p.u_ts)[d]);
        float s = to_f32((dl + t * p.delta_ts)[d]) + bias;
        const Pack<T, 4> bv = piece(B + t * p.B_ts), cv = piece(C + t * p.C_ts);
        const float zv = p.z ? to_f32((z + t * p.z_ts)[d]) : 0.0f;
        if (p.softplus) s = softplus(s);
        float acc = advance(s, s * uv, bv, cv);
        acc = fmaf(skip, uv, lanes_sum<W>(acc));
        if (p.z) acc *= silu<T>(zv);
        if (part == 0) (y + t * p.channels)[d] = from_f32<T>(acc);
        if (p.state_out && t == j) *reinterpret_cast<f32x4 *>(p.state_out + at) = h;
    };
    if constexpr (ONE) {
        if (len > 0) one(0);
    } else {
        int t = 0;
        if constexpr (W >= 4) {
            const int q = tid & 3;
            for (; t < len; t += 4) {
                if (t + 4 > len || (j >= t && j < t + 4)) {
                    for (int k = t; k < min(t + 4, len); ++k) one(k);
                    continue;
                }
                const float uv = to_f32((u + (int64_t)(t + q) * p.u_ts)[d]);
                float s = to_f32((dl + (int64_t)(t + q) * p.delta_ts)[d]) + bias;
                const float zv = p.z ? to_f32((z + (int64_t)(t + q) * p.z_ts)[d]) : 0.0f;
                Pack<T, 4> bv[4], cv[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bv[k] = piece(B + (int64_t)(t + k) * p.B_ts);
                    cv[k] = piece(C + (int64_t)(t + k) * p.C_ts);
                }
                if (p.softplus) s = softplus(s);
                const float du = s * uv;
                const float acc[4] = {advance(of_quad<0>(s), of_quad<0>(du), bv[0], cv[0]),
                                      advance(of_quad<1>(s), of_quad<1>(du), bv[1], cv[1]),
                                      advance(of_quad<2>(s), of_quad<2>(du), bv[2], cv[2]),
                                      advance(of_quad<3>(s), of_quad<3>(du), bv[3], cv[3])};
                float r = fmaf(skip, uv, lanes_sum4<W>(acc));
                if (p.z) r *= silu<T>(zv);
                if (part < 4) (y + (int64_t)(t + q) * p.channels)[d] = from_f32<T>(r);
            }
        }
        for (; t < len; ++t) one(t);
    }
    if (p.final_state) *reinterpret_cast<f32x4 *>(p.final_state + at) = h;
}

// Calls up to this many tokens run without tiles (us by steps / by tiles: 64
// sequences of 5120 channels 8 tokens 25 / 53, 16 tokens 41 / 57, 24 tokens 57 /
// 60, 32 tokens 74 / 67; one sequence 16 tokens 6.1 / 6.5, 24 tokens 7.7 / 7.1).
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
        if (p.seqlen <= 1) scan_steps_kernel<T, N, true><<<grid, kThreads, 0, stream>>>(p);
        else scan_steps_kernel<T, N, false><<<grid, kThreads, 0, stream>>>(p);
        return hipGetLastError();
    }
    return p.group_channels % (int)(16 / sizeof(T)) == 0 ? run_tiles<T, N, false>(p, stream) : run_tiles<T, N, true>(p, stream);
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
    // Workgroups of an unsplit call; a compute unit holds three (two with 32
    // or more states, by LDS and registers).  Ranges double the work and cost
    // another launch and prologue, some 6 us: with one workgroup on a compute
    // unit taking 0.109 us per token and three of them 0.209 (N 16), they pay
    // from T (1 - wgs / 224) = 55 tokens on, fewer with more states.  (us
    // without / with them: 24 workgroups, 200 tokens 27 / 16, 4093 tokens 438 /
    // 61; 80, 100 tokens 15.5 / 13.8, 2048 tokens 223 / 115; 192, 100 tokens
    // 16 / 22; 160, 2048 tokens 228 / 190 with four ranges, 278 with two; 320,
    // 2048 tokens 304 / 348 with two: hence room for at least four.)  Whole
    // tiles may leave three of the four or five asked for, with 129 to 288
    // tokens on 86 to 181 workgroups; three cost 0.9 to 1.11 of a call without
    // ranges (us with three / none: N 16, 160 workgroups 192 tokens 28 / 25, 288
    // tokens 37.5 / 36; 128 workgroups 288 tokens 34 / 35; N 64, 128 workgroups
    // 160 tokens 55 / 49.5, 288 tokens 77 / 86).
    const int64_t tiles = (p.group_channels + kChannels - 1) / kChannels;
    const int64_t wgs = tiles * p.ngroups * p.batch, held = (p.dstate >= 32 ? 2 : 3) * (int64_t)256;
    const int64_t want = std::min(held / wgs, (p.seqlen + kTile - 1) / kTile);
    if (want < 4 || p.seqlen * (224 - wgs) * p.dstate < (int64_t)3 << 16) return;
    p.range_len = ((p.seqlen + want - 1) / want + kTile - 1) / kTile * kTile;
    p.ranges = (int)((p.seqlen + p.range_len - 1) / p.range_len);
}

hipError_t launch_selective_scan(const SelectiveParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? by_state<bf16>(p, stream) : by_state<float>(p, stream);
}

}  // namespace ssd
