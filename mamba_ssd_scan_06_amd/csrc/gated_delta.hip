// Gated delta rule token by token, for calls of a few tokens (a decode step,
// the verification of drafts):
//
//     S = e^g S;   r = v - S k;   S += beta r k';   y = scale S q
//
// Every row p of S [P,N] is on its own, so a workgroup takes 32 rows of one
// (sequence, head), or 64, with 8 lanes per row and the row in their registers: the
// state is read once and written once, 16 bytes per lane, and S k and S q are
// joined over a row's lanes by three lane exchanges.  k, q (fp32, normalised
// where asked), v, e^g and beta of 8 tokens at a time are laid out in LDS by the
// whole workgroup; the loads of the state are issued before that.
//
// Bound by the states' traffic: one token of 64 sequences (32 heads, N and P 128)
// 49 us, 5.5 TB/s; nine with the accepted state 91 us, 4.5 TB/s, where the vector
// instructions are 55% of the time; one token of one sequence 4.9 us, a launch.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kRows = 32;    // rows of a workgroup, of each of a lane's R
constexpr int kLanes = 8;    // lanes of a row
constexpr int kBlock = 8;    // tokens laid out at a time
constexpr float kNormEps = 1e-6f;

// Sum over the 8 lanes of a row, the same value in all of them.
template <int CTRL>
__device__ __forceinline__ float lane_moved(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum8(float v) {
    v += lane_moved<0xB1>(v);   // quad_perm 1,0,3,2
    v += lane_moved<0x4E>(v);   // quad_perm 2,3,0,1
    v += lane_moved<0x141>(v);  // row_half_mirror: the other quad of the eight
    return v;
}

// M: 16-byte pieces of a row per lane; piece m of lane l holds n = 4 (8 m + l)
// and the three after it.
template <typename T, int M, int R>
__global__ __launch_bounds__(kRows * kLanes) void delta_tokens(DeltaParams p) {
    constexpr int NP = M * kLanes * 4;  // N, rounded up to whole pieces of all lanes
    __shared__ __attribute__((aligned(16))) float ks[kBlock][NP], qs[kBlock][NP];
    __shared__ float vs[kBlock][R * kRows], ys[kBlock][R * kRows], decay[kBlock], share[kBlock];
    const int tid = threadIdx.x, lane = tid & (kLanes - 1), row = tid / kLanes, wave = tid >> 6;
    const int slices = (p.headdim + R * kRows - 1) / (R * kRows);
    const unsigned item = blockIdx.x / (unsigned)slices, slice = blockIdx.x - item * (unsigned)slices;
    const unsigned b = item / (unsigned)p.nheads, h = item - b * (unsigned)p.nheads;
    const int N = p.dstate, pieces = N / 4, p0 = (int)slice * R * kRows, rows = min(R * kRows, p.headdim - p0);
    const int64_t s_off = ((int64_t)item * p.headdim + p0 + row) * N + 4 * lane;  // of the first row

    f32x4 s[R][M];
    auto store_state = [&](float *to) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (row + r * kRows < rows)
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (kLanes * m + lane < pieces)
                        __builtin_nontemporal_store(
                            s[r][m], reinterpret_cast<f32x4 *>(to + s_off + (int64_t)r * kRows * N + 4 * kLanes * m));
    };
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            s[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (p.init_state && row + r * kRows < rows && kLanes * m + lane < pieces)
                s[r][m] = __builtin_nontemporal_load(
                    reinterpret_cast<const f32x4 *>(p.init_state + s_off + (int64_t)r * kRows * N + 4 * kLanes * m));
        }
    int64_t at = -2;  // the accepted index
    if (p.state_out) {
        at = min(max((int64_t)p.state_out_idx[b], (int64_t)-1), p.seqlen - 1);
        if (at < 0) store_state(p.state_out);
    }

    const int group = (int)h / p.heads_per_group;
    for (int64_t t0 = 0; t0 < p.seqlen; t0 += kBlock) {
        const int count = (int)min((int64_t)kBlock, p.seqlen - t0);
        // k and q: a wave per row of either, two per token.
        for (int r = wave; r < 2 * count; r += kRows * kLanes / 64) {
            const int t = r >> 1, is_q = r & 1;
            const T *src = is_q ? reinterpret_cast<const T *>(p.q) + b * p.q_bs + (t0 + t) * p.q_ts
                                : reinterpret_cast<const T *>(p.k) + b * p.k_bs + (t0 + t) * p.k_ts;
            src += (int64_t)group * N;
            float v[(NP + 63) / 64], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < (NP + 63) / 64; ++i) {
                const int n = 64 * i + (tid & 63);
                v[i] = n < N ? to_f32(src[n]) : 0.0f;
                sum = fmaf(v[i], v[i], sum);
            }
            float f = 1.0f;
            if (p.l2norm) {
                for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
                f = 1.0f / sqrtf(sum + kNormEps);
            }
            if (is_q) f *= p.scale;
            float *dst = is_q ? qs[t] : ks[t];
#pragma unroll
            for (int i = 0; i < (NP + 63) / 64; ++i) {
                const int n = 64 * i + (tid & 63);
                if (n < NP) dst[n] = v[i] * f;
            }
        }
        {
            const int t = tid / kRows;  // kBlock x kRows values by as many threads
#pragma unroll
            for (int r = tid & (kRows - 1); r < R * kRows; r += kRows)
                if (t < count && r < rows)
                    vs[t][r] = to_f32((reinterpret_cast<const T *>(p.v) + b * p.v_bs + (t0 + t) * p.v_ts)[(int64_t)h * p.headdim + p0 + r]);
            if (tid < count) {
                decay[tid] = p.g ? expf(p.g[b * p.g_bs + (t0 + tid) * p.g_ts + h]) : 1.0f;
                share[tid] = p.beta[b * p.beta_bs + (t0 + tid) * p.beta_ts + h];
            }
        }
        __syncthreads();
        for (int t = 0; t < count; ++t) {
            const float a = decay[t];
            float dot[R] = {}, out[R] = {}, u[R];
            f32x4 k[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                k[m] = *reinterpret_cast<const f32x4 *>(&ks[t][4 * (kLanes * m + lane)]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[r][m][i] *= a;
                        dot[r] = fmaf(s[r][m][i], k[m][i], dot[r]);
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) u[r] = share[t] * (vs[t][row + r * kRows] - sum8(dot[r]));
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const f32x4 q = *reinterpret_cast<const f32x4 *>(&qs[t][4 * (kLanes * m + lane)]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[r][m][i] = fmaf(u[r], k[m][i], s[r][m][i]);
                        out[r] = fmaf(s[r][m][i], q[i], out[r]);
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                out[r] = sum8(out[r]);
                if (lane == 0) ys[t][row + r * kRows] = out[r];
            }
            if (t0 + t == at) store_state(p.state_out);
        }
        __syncthreads();
        {
            const int t = tid / kRows;
#pragma unroll
            for (int r = tid & (kRows - 1); r < R * kRows; r += kRows)
                if (t < count && r < rows)
                    (reinterpret_cast<T *>(p.y) + ((int64_t)b * p.seqlen + t0 + t) * p.nheads * p.headdim)[(int64_t)h * p.headdim + p0 + r] =
                        from_f32<T>(ys[t][r]);
        }
        // The next block's first barrier stands between these reads of ys and
        // its writes.
    }
    if (p.final_state) store_state(p.final_state);
}

template <typename T, int M>
hipError_t launch(const DeltaParams &p, hipStream_t stream) {
    // Two rows per lane halve the reads of k and q from LDS, where enough
    // workgroups remain: N and P 128, 32 heads, 9 tokens of 8, 16 and 64 sequences
    // 14.0, 27.3 and 101 us with one, 15.2, 21.9 and 90 with two.  N beyond 160 has
    // too many registers (256, 16 heads, 16 tokens of 32 sequences: 129 and 142);
    // for 2 tokens of 64 sequences only the states' traffic counts, which more waves
    // carry better (70 and 75; 16 sequences 18.6 and 16.7).  Rows that 64 leave empty
    // cost as much as others: N 128, 9 tokens of 64 sequences, P 16 and 32 24.0 and
    // 25.7 us with one, 30.2 and 32.1 with two, P 80 and 96 68 and 70, 72 and 74, but
    // P 48 50 and 36, P 144 and 160 107 and 101.  So never where they are half, and
    // up to a quarter, or a third where the workgroups are few (P 80, 16 sequences
    // 20.8 and 18.8).
    const int slices = (p.headdim + kRows - 1) / kRows, wide = (p.headdim + 2 * kRows - 1) / (2 * kRows);
    const int64_t pairs = p.batch * p.nheads * wide;
    const bool fills = slices > 1 && (8 * wide <= 5 * slices || pairs < 2048);
    const bool two = M <= 5 && fills && pairs >= 1024 && (p.seqlen >= 4 || pairs < 4096);
    const int rows = two ? 2 * kRows : kRows;
    const unsigned grid = (unsigned)(p.batch * p.nheads * ((p.headdim + rows - 1) / rows));
    if constexpr (M <= 5)
        if (two) {
            delta_tokens<T, M, 2><<<grid, kRows * kLanes, 0, stream>>>(p);
            return hipGetLastError();
        }
    delta_tokens<T, M, 1><<<grid, kRows * kLanes, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t run(const DeltaParams &p, hipStream_t stream) {
    switch ((p.dstate + 31) / 32) {
        case 1: return launch<T, 1>(p, stream);
        case 2: return launch<T, 2>(p, stream);
        case 3: return launch<T, 3>(p, stream);
        case 4: return launch<T, 4>(p, stream);
        case 5: return launch<T, 5>(p, stream);
        case 6: return launch<T, 6>(p, stream);
        case 7: return launch<T, 7>(p, stream);
        default: return launch<T, 8>(p, stream);
    }
}

}  // namespace

hipError_t launch_delta_tokens(const DeltaParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
