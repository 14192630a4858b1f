// Gated delta rule in chunks of 32 tokens, for prompts.
//
// With Gam_i the sum of g from the chunk's first token to token i, S the state
// that enters the chunk and kr, qr the factors that normalise and scale keys and
// queries, the chunk's updates u (S_t = ... + kr_t u_t k_t') solve
//
//     u_i + beta_i sum_{j<i} e^{Gam_i-Gam_j} kr_i kr_j (k_i.k_j) u_j
//         = beta_i (v_i - e^{Gam_i} kr_i S k_i),
//
// so U = Tb X with Tb = (1 + A)^-1 diag(beta) and X_i = v_i - a_i S k_i, and
//
//     y_i = c_i S q_i + sum_{j<=i} Pm_ij u_j,  Pm_ij = qr_i kr_j e^{Gam_i-Gam_j} q_i.k_j
//     S'  = e^{Gam_C} S + sum_j d_j u_j k_j',  a = e^{Gam} kr, c = e^{Gam} qr, d = e^{Gam_C-Gam} kr.
//
// Two launches (four where the sequence is cut into ranges, see delta_ranges).
// delta_prepare takes a wave per (sequence, chunk, head), all of
// them at once, and leaves Tb and Pm in the workspace in the order in which the
// matrix cores read them, with the tables a, c, d.  delta_chunks walks the chunks
// of a (sequence, head) in order.  There a wave owns 16 rows p of the state and
// all of N, as S' tiles [n, p] in its accumulators: a result tile (rows 4 (l/16)
// + r, column l%16 = p) is the next product's operand as it stands, so nothing
// passes between waves and only the operands that they share (k, q, v, Tb, Pm)
// go through LDS, one chunk ahead.
//
// States, X and U are fp32 and enter the products as sums of bf16 terms: three
// hold all 24 bits of the fraction, and of the products of two such sums those
// below 2^-24 of the first are left out.  bf16 inputs are one term, fp32 ones
// three.  This is 3 to 6 products of the bf16 rate, which is 16 times the fp32
// rate.  Tb X and Pm U of bf16 calls, where neither side is a bf16 input, are fp32
// products instead: twice the matrix cores' time of six products of terms, but no
// vector instructions for X's and U's terms, and two thirds of the tables' bytes.
//
// 8 x 2048 tokens of 32 heads (N and P 128, 8 groups, bf16) take 237 us: the
// preparation 40, bound by its 186 MB of reads and tables (4.6 TB/s), the chunks
// 196, in which the matrix cores are 66% busy with 116 products per wave and chunk
// (24 of them fp32, of twice the cycles) and the vector instructions (257) 30%.  The
// two hardly overlap: both waves of a SIMD walk the same phases.
#include <math.h>

#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int C = kDeltaChunk;   // 32 tokens
constexpr int kThreads = 256;    // four waves
constexpr int kSlice = 64;       // rows of the state of a workgroup, 16 per wave
constexpr float kNormEps = 1e-6f;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2), may_alias));

template <typename T> constexpr int kIn = sizeof(T) == 2 ? 1 : 3;   // terms of an input

// What delta_prepare leaves per (sequence, chunk, head), in bytes: Tb, Pm, then
// the tables.  bf16: Tb and Pm in fp32, tiles 00, 10 and 11, four values of each
// per lane.  fp32: their terms, by row tile (the upper one needs the first 16
// tokens only: half fragments) and term.
template <typename T>
struct Pack32 {
    static constexpr bool kTerms = sizeof(T) == 4;
    static constexpr int kValue = kTerms ? 6 : 4;  // bytes
    static constexpr int kT0 = 0, kT1 = kT0 + 64 * 4 * kValue, kP0 = kT1 + 64 * 8 * kValue, kP1 = kP0 + 64 * 4 * kValue,
                         kTab = kP1 + 64 * 8 * kValue, kUsed = kTab + 512;
    // The direct copies' two instructions of 1 KB per wave.
    static constexpr int kBytes = kTerms ? kUsed : 8 * 1024;
    // floats of the tables
    static constexpr int kA = 0, kC = 32, kD = 64, kEnd = 96;
};
constexpr int kAtFloats = 36;  // the accepted index's weights [32] and decay, per (sequence, head)

// The least log decay that enters the sums of a chunk.  Its exponential is 0 (of
// anything below -104), and so is that of any sum with it unless more than 65000
// follows; but sums of 32 stay below 2^22 (times log2 e), where two floats, and the
// double before them, hold the differences of later tokens to 2^-27.  Without it
// -1e14 would swallow the decays after it, and an infinity make them NaN.
constexpr float kLeastDecay = -65536.0f;

// A sum of log decays in two floats, its rounding and what that left: sums of a
// chunk may be large where their differences are small.
struct TwoFloats {
    float hi, lo;
};
__device__ __forceinline__ TwoFloats two_floats(double v) {
    const float hi = (float)v;
    return {hi, (float)(v - (double)hi)};
}
// 2^(a - b), for sums below 2^22 in size: off by |a - b| 2^-24 and 2^-26 of itself
// beside the hardware exponential's unit.  Where a <= b the first is below 2^-24
// absolutely.
__device__ __forceinline__ float exp2_diff(const TwoFloats &a, const TwoFloats &b) {
    return exp2_hw((a.hi - b.hi) + (a.lo - b.lo));
}

// v as a sum of N bf16 terms, each the next 8 bits of the fraction (cut off, so
// that three terms are v itself).  A pair of
// values takes one byte permutation per term and an and and a subtraction per
// value between terms; rounding with v_cvt_pk_bf16_f32 costs as many and half of
// them at twice the time.
template <int N, int LEN, typename V>
__device__ __forceinline__ void split(const float (&v)[LEN], V (&t)[N]) {
    uint32_t w[N][LEN / 2];
#pragma unroll
    for (int i = 0; i < LEN; i += 2) {
        float lo = v[i], hi = v[i + 1];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t l = __builtin_bit_cast(uint32_t, lo), h = __builtin_bit_cast(uint32_t, hi);
            w[k][i / 2] = __builtin_amdgcn_perm(h, l, 0x07060302u);
            if (k + 1 < N) {
                lo -= __builtin_bit_cast(float, l & 0xffff0000u);
                hi -= __builtin_bit_cast(float, h & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) __builtin_memcpy(&t[k], w[k], sizeof(V));
}

__device__ __forceinline__ f32x4 mfma(const bf16x8 &a, const bf16x8 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(const bf16x4 &a, const bf16x4 &b, const f32x4 &c) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
}
// acc += (sum of a's terms) (sum of b's terms) without the products below the
// last bit kept, the smallest first.
template <int TA, int TB, typename V, int NA, int NB>
__device__ __forceinline__ void mma_terms(const V (&a)[NA], const V (&b)[NB], f32x4 &acc) {
    static_assert(TA <= NA && TB <= NB, "terms");
    constexpr int K = TA > TB ? TA : TB;
#pragma unroll
    for (int s = K - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < TA; ++i)
            if (s - i >= 0 && s - i < TB) acc = mfma(a[i], b[s - i], acc);
}

// ------------------------------------------------------------------ prepare
template <typename T> __device__ __forceinline__ void load_frag(Frag<T> &f, const T *p);
template <> __device__ __forceinline__ void load_frag<bf16>(Frag<bf16> &f, const bf16 *p) {
    f.v = __builtin_bit_cast(bf16x8, load_words(p));
}
template <> __device__ __forceinline__ void load_frag<float>(Frag<float> &f, const float *p) {
    f.lo = __builtin_bit_cast(f32x4, load_words(p));
    f.hi = __builtin_bit_cast(f32x4, load_words(p + 4));
}
__device__ __forceinline__ float squares(const Frag<bf16> &f, float s) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const bf16x2 v = {f.v[i], f.v[i + 1]};
        s = __builtin_amdgcn_fdot2_f32_bf16(v, v, s, false);
    }
    return s;
}
__device__ __forceinline__ float squares(const Frag<float> &f, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(f.hi[i], f.hi[i], fmaf(f.lo[i], f.lo[i], s));
    return s;
}
__device__ __forceinline__ f32x4 mma_f32_16(const f32x4 &a, const f32x4 &b, f32x4 acc) {
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
    return acc;
}

struct WaveTables {
    float hi[C], lo[C];  // Gam_i log2 e
    float beta[C], kr[C], qr[C];
    float at[2][16][20];  // A's diagonal blocks, transposed: [j][m]; rows padded
    float tb[2][16][20];  // their inverses, row-major
};

// Orders a wave's own accesses to LDS (which the hardware takes in order).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave per (b, chunk, p.prepare_heads heads of a group), which have their keys,
// queries, these products and norms in common.  Every 16 x 16 tile is computed transposed, so
// that lane l holds row i = l%16 and columns j = 4 (l/16) + r: the layout in which
// delta_chunks feeds it to the matrix cores.  The inverse takes the two diagonal
// blocks by substitution (a lane per row: t_j = [j = i] - sum_{m>j} t_m A_mj) and
// joins them, -T11 A10 T00, by fp32 products.
template <typename T, int NB>
__global__ __launch_bounds__(kThreads) void delta_prepare(DeltaParams p) {
    __shared__ WaveTables tables[kThreads / 64];
    const int uwave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    WaveTables &w = tables[uwave];
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const unsigned parts = (unsigned)(p.nheads / p.prepare_heads);
    const unsigned items = (unsigned)(p.batch * p.nchunks) * parts, item = blockIdx.x * (kThreads / 64) + uwave;
    if (item >= items) return;
    const unsigned bc = item / parts, h0 = (item - bc * parts) * (unsigned)p.prepare_heads;
    const unsigned b = bc / (unsigned)p.nchunks, c = bc - b * (unsigned)p.nchunks;
    const int64_t t0 = (int64_t)c * C;
    const int left = (int)min(p.seqlen - t0, (int64_t)C);  // tokens of this chunk
    const int group = (int)h0 / p.heads_per_group;

    // Keys and queries: rows of token tile I in lanes i16.
    const T *kbase = reinterpret_cast<const T *>(p.k) + b * p.k_bs + t0 * p.k_ts + (int64_t)group * p.dstate;
    const T *qbase = reinterpret_cast<const T *>(p.q) + b * p.q_bs + t0 * p.q_ts + (int64_t)group * p.dstate;
    Frag<T> kf[NB][2], qf[NB][2];
#pragma unroll
    for (int I = 0; I < 2; ++I) {
        const int t = min(16 * I + i16, left - 1);
        const T *kr = kbase + t * p.k_ts + 8 * g, *qr = qbase + t * p.q_ts + 8 * g;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            const bool in = 32 * kb + 8 * g < p.dstate;  // else the row's first piece, made zero below
            load_frag<T>(kf[kb][I], kr + (in ? 32 * kb : -8 * g));
            load_frag<T>(qf[kb][I], qr + (in ? 32 * kb : -8 * g));
        }
    }

    // Log decay and beta of token `lane` of head h; past the end nothing is
    // written (beta 0) and nothing decays.
    auto token = [&](unsigned h, float &gt, float &bt) {
        gt = bt = 0.0f;
        if (lane < left) {
            if (p.g) gt = p.g[b * p.g_bs + (t0 + lane) * p.g_ts + h];
            gt = gt < kLeastDecay ? kLeastDecay : gt;  // a NaN stays one
            bt = p.beta[b * p.beta_bs + (t0 + lane) * p.beta_ts + h];
        }
    };
    float g_next, beta_next;
    token(h0, g_next, beta_next);

    // Products of keys with keys and queries: tile (I, J) = lanes (i in I, j in J).
    f32x4 kk[3] = {}, qk[3] = {};  // tiles 00, 10, 11
    float ksq[2] = {0.f, 0.f}, qsq[2] = {0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
        if (32 * NB > p.dstate && 32 * kb + 8 * g >= p.dstate)
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                kf[kb][I].zero();
                qf[kb][I].zero();
            }
        const Frag<T>(&k)[2] = kf[kb];
        const Frag<T>(&q)[2] = qf[kb];
        mma(k[0], k[0], kk[0]);
        mma(k[0], k[1], kk[1]);
        mma(k[1], k[1], kk[2]);
        mma(k[0], q[0], qk[0]);
        mma(k[0], q[1], qk[1]);
        mma(k[1], q[1], qk[2]);
        if (p.l2norm)
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                ksq[I] = squares(k[I], ksq[I]);
                qsq[I] = squares(q[I], qsq[I]);
            }
    }
#pragma unroll
    for (int I = 0; I < 2; ++I) {
        float kr = 1.0f, qr = p.scale;
        if (p.l2norm) {
#pragma unroll
            for (int m = 16; m < 64; m <<= 1) {
                ksq[I] += __shfl_xor(ksq[I], m);
                qsq[I] += __shfl_xor(qsq[I], m);
            }
            kr = 1.0f / sqrtf(ksq[I] + kNormEps);
            qr *= 1.0f / sqrtf(qsq[I] + kNormEps);
        }
        if (g == 0) {
            w.kr[16 * I + i16] = kr;
            w.qr[16 * I + i16] = qr;
        }
    }

    for (unsigned h = h0;;) {
        double gam = (double)g_next * 1.4426950408889634;
#pragma unroll
        for (int m = 1; m < C; m <<= 1) {
            const double o = __shfl_up(gam, m);
            if (lane >= m) gam += o;
        }
        const TwoFloats mine = two_floats(gam);
        if (lane < C) {
            w.hi[lane] = mine.hi;
            w.lo[lane] = mine.lo;
            w.beta[lane] = beta_next;
        }
        if (h + 1 < h0 + p.prepare_heads) token(h + 1, g_next, beta_next);
        wave_sync();

        // A and Pm.
        float pm[3][4];
        f32x4 a10, bj[2];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int I = (k + 1) / 2, J = k / 2, i = 16 * I + i16, j0 = 16 * J + 4 * g;
            const TwoFloats ci = {w.hi[i], w.lo[i]};
            const float bi = w.beta[i] * w.kr[i], qi = w.qr[i];
            const f32x4 hj = *reinterpret_cast<const f32x4 *>(&w.hi[j0]), lj = *reinterpret_cast<const f32x4 *>(&w.lo[j0]),
                        kj = *reinterpret_cast<const f32x4 *>(&w.kr[j0]);
            bj[J] = *reinterpret_cast<const f32x4 *>(&w.beta[j0]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = exp2_diff(ci, {hj[r], lj[r]}) * kj[r];
                pm[k][r] = j0 + r <= i ? qi * e * qk[k][r] : 0.0f;
                const float a = j0 + r < i ? bi * e * kk[k][r] : 0.0f;
                if (k == 1) a10[r] = a;
                else w.at[I][4 * g + r][i16] = a;
            }
        }
        wave_sync();
        {
            const int blk = g & 1;
            float t[16];
#pragma unroll
            for (int j = 15; j >= 0; --j) {
                float s = j == i16 ? 1.0f : 0.0f;
#pragma unroll
                for (int m = 15; m > j; --m) s = fmaf(-t[m], w.at[blk][j][m], s);
                t[j] = s;
            }
            if (g < 2)
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<f32x4 *>(&w.tb[blk][i16][j]) = f32x4{t[j], t[j + 1], t[j + 2], t[j + 3]};
        }
        wave_sync();
        f32x4 tt[3];
        tt[0] = *reinterpret_cast<const f32x4 *>(&w.tb[0][i16][4 * g]);
        tt[2] = *reinterpret_cast<const f32x4 *>(&w.tb[1][i16][4 * g]);
        f32x4 t00t;
#pragma unroll
        for (int r = 0; r < 4; ++r) t00t[r] = w.tb[0][4 * g + r][i16];
        const f32x4 prod = mma_f32_16(a10, t00t, f32x4{0.f, 0.f, 0.f, 0.f});  // (A10 T00)[m][j]: lane j, rows m
        const f32x4 joined = mma_f32_16(prod, tt[2], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < 4; ++r) tt[1][r] = -joined[r];

        typedef Pack32<T> L;
        const int64_t bh = (int64_t)b * p.nheads + h;
        char *out = p.pack + ((int64_t)bc * p.nheads + h) * L::kBytes;
        float tv[3][4];
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) tv[k][r] = tt[k][r] * bj[k / 2][r];
        [[maybe_unused]] auto put = [&](const float (&lo)[4], const float (&hi)[4], int off) {
            const float both[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            bf16x8 f[3];
            split(both, f);
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<bf16x8 *>(out + off + (k * 64 + lane) * 16) = f[k];
        };
        [[maybe_unused]] auto put_half = [&](const float (&v)[4], int off) {
            bf16x4 f[3];
            split(v, f);
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<bf16x4 *>(out + off + (k * 64 + lane) * 8) = f[k];
        };
        if constexpr (L::kTerms) {
            put_half(tv[0], L::kT0);
            put(tv[1], tv[2], L::kT1);
            put_half(pm[0], L::kP0);
            put(pm[1], pm[2], L::kP1);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                *reinterpret_cast<f32x4 *>(out + L::kT0 + (k * 64 + lane) * 16) = f32x4{tv[k][0], tv[k][1], tv[k][2], tv[k][3]};
                *reinterpret_cast<f32x4 *>(out + L::kP0 + (k * 64 + lane) * 16) = f32x4{pm[k][0], pm[k][1], pm[k][2], pm[k][3]};
            }
        }
        float *tab = reinterpret_cast<float *>(out + L::kTab);
        if (lane < C) {
            const TwoFloats zero = {0.f, 0.f}, end = {w.hi[C - 1], w.lo[C - 1]};
            const float e = exp2_diff(mine, zero), kr = w.kr[lane];
            tab[L::kA + lane] = e * kr;
            tab[L::kC + lane] = e * w.qr[lane];
            tab[L::kD + lane] = exp2_diff(end, mine) * kr;
            if (lane == 0) tab[L::kEnd] = exp2_diff(end, zero);
        }
        if (p.state_out) {
            const int64_t at = min(max((int64_t)p.state_out_idx[b], (int64_t)-1), p.seqlen - 1) - t0;
            if (at >= 0 && at < C && lane < C) {
                float *to = p.at_tables + bh * kAtFloats;
                const TwoFloats ce = {w.hi[(int)at], w.lo[(int)at]};
                to[lane] = lane <= (int)at ? exp2_diff(ce, mine) * w.kr[lane] : 0.0f;
                if (lane == 0) to[C] = exp2_diff(ce, {0.f, 0.f});
            }
        }
        if (++h == h0 + p.prepare_heads) break;
        wave_sync();  // the next head's tables
    }
}
// ------------------------------------------------------------------- chunks
// LDS of a chunk.  Rows of keys and queries (4 NB pieces of 16 bytes) are not
// padded, so that a copy may fill them in order; instead the pieces of row r
// stand at piece ^ key_swz(r).  A read of 16 bytes is served in turns of lanes 0-3,
// 12-15, 20-23 and 24-27, then 4-11, 16-19 and 28-31, and the same of the upper
// half; the negative sign sets the rows that lanes 0-15 and 16-31 read of such a
// turn apart (counters: a plain r / 4 makes every read wait for two).  Transposed
// reads take 8 bytes of each piece, which meets half of the banks twice.
template <int NB>
__device__ __forceinline__ int key_swz(int r) {
    int s = -(r >> 2) & 3;                           // rows that are a multiple of 256 bytes apart
    if constexpr (NB % 4 == 0) s |= 4 * (r & 3);
    else if constexpr (NB % 2 == 0) s |= 4 * ((r >> 1) & 1);
    return s;
}
// v: rows of 64 values; bf16 ones are read transposed, two pieces of four rows.
template <typename T>
__device__ __forceinline__ int v_swz(int r) {
    return sizeof(T) == 2 ? 2 * ((r >> 1) & 3) : 0;
}
template <typename T, int NB, bool OUT>
struct Queries {
    alignas(16) bf16 q[kIn<T>][C][32 * NB];
};
template <typename T, int NB>
struct Queries<T, NB, false> {};  // without outputs there is room for more workgroups
template <typename T, int NB, bool OUT>
struct Buffer : Queries<T, NB, OUT> {
    static constexpr int kPlane = 32 * NB;           // elements of a row of keys or queries
    static constexpr int kVRow = kSlice + (sizeof(T) == 2 ? 0 : 8);
    alignas(16) bf16 k[kIn<T>][C][kPlane];
    alignas(16) T v[C][kVRow];
    alignas(16) char pack[Pack32<T>::kBytes];
};

// What a thread carries from global memory to LDS, one chunk ahead.
template <typename T, int NB, bool OUT>
struct Carry {
    static constexpr int VEC = 16 / sizeof(T), WORDS = 8 / VEC;  // 16-byte words of 8 elements
    static constexpr int kPackWords = (Pack32<T>::kBytes / 16 + kThreads - 1) / kThreads;
    static constexpr int kKeys = OUT ? NB : (NB + 1) / 2;
    u32x4 kq[kKeys][WORDS], v[WORDS], pack[kPackWords];
};

// WAVES: waves per SIMD to leave registers for (two keep the accumulators in
// the ordinary registers too).  DIRECT: bf16 rows of 16-byte alignment, which the
// buffer loads that write LDS by themselves take; other rows pass through
// registers.  OUT: outputs are computed (and the chunks of one range are walked
// from its entering state); without, the first pass over the ranges: each leaves
// its final state from a zero start (the first one from init_state) and, in
// further slices of rows that start as the unit matrix with v = 0, the map M of
// the state that enters it (S_end = S_begin M + that final state).
template <typename T, int NB, int BUFS, int WAVES, bool DIRECT, bool OUT>
__global__ __launch_bounds__(kThreads, WAVES) void delta_chunks(DeltaParams p) {
    typedef Pack32<T> L;
    typedef Buffer<T, NB, OUT> Buf;
    typedef Carry<T, NB, OUT> Regs;
    constexpr int NI = kIn<T>;
    static_assert(!DIRECT || (sizeof(T) == 2 && BUFS == 2 && L::kBytes == 8 * 1024), "direct copies");
    // Two objects, so that the compiler knows reads of one apart from the copies
    // into the other and does not make them wait.
    __shared__ Buf buf0;
    __shared__ std::conditional_t<BUFS == 2, Buf, char> buf1_;
    Buf &buf1 = *reinterpret_cast<Buf *>(BUFS == 2 ? (void *)&buf1_ : (void *)&buf0);

    // Consecutive items (the slices of a head, the heads of a group) on one XCD.
    const unsigned xcd = blockIdx.x % 8, whole = gridDim.x / 8, more = gridDim.x % 8;
    const unsigned item = xcd * whole + min(xcd, more) + blockIdx.x / 8;
    // An item is a slice of rows of a (sequence, range, head), in this order.
    const int v_slices = (p.headdim + kSlice - 1) / kSlice;
    const int slices = OUT ? v_slices : v_slices + (p.dstate + kSlice - 1) / kSlice;
    const unsigned brh = item / (unsigned)slices, br = brh / (unsigned)p.nheads, h = brh - br * (unsigned)p.nheads;
    const unsigned ranges = (unsigned)(OUT ? p.ranges : p.ranges - 1), b = br / ranges, range = br - b * ranges;
    const unsigned bh = b * (unsigned)p.nheads + h;
    const int slice = (int)(item - brh * (unsigned)slices);
    const bool map = !OUT && slice >= v_slices;
    if (map && range == 0) return;  // nothing enters the first range but init_state
    const int slice0 = (map ? slice - v_slices : slice) * kSlice, all_rows = map ? p.dstate : p.headdim;
    // This range's tokens: the first, and how many.
    const int64_t first = (int64_t)range * p.range_chunks * C;
    const int tokens = (int)min(p.range_chunks * C, p.seqlen - first);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i16 = lane & 15, g = lane >> 4;
    const int N = p.dstate, p0 = slice0 + 16 * wave;
    const bool live = p0 < all_rows;  // whole waves only: both sizes are multiples of 16
    const int group = (int)h / p.heads_per_group;

    const T *kbase = reinterpret_cast<const T *>(p.k) + b * p.k_bs + first * p.k_ts + (int64_t)group * N;
    const T *qbase = reinterpret_cast<const T *>(p.q) + b * p.q_bs + first * p.q_ts + (int64_t)group * N;
    const T *vbase = reinterpret_cast<const T *>(p.v) + b * p.v_bs + first * p.v_ts + (int64_t)h * p.headdim + (map ? 0 : slice0);
    const int v_cols = map ? 0 : min(kSlice, p.headdim - slice0);  // a map has no v: zeros
    const char *packs = p.pack + (((int64_t)b * p.nchunks + first / C) * p.nheads + h) * L::kBytes;
    const int64_t pack_stride = (int64_t)p.nheads * L::kBytes;
    // Direct copies: a wave instruction fills 64 consecutive 16-byte pieces of
    // LDS, each lane from an offset of its own into the chunk's rows.  Columns
    // past N and rows past the end lie beyond the buffer, which reads as 0.  A
    // wave issues NB of the keys' and queries' 4 NB instructions, one of v's
    // four and two of the eight of Tb, Pm and the tables; only the buffers'
    // bases move, in scalar registers.  They are spread over the steps of the
    // chunk before (fetch_step): the texture path takes 64 bytes a cycle, and a
    // wave that issues all of its copies at once waits for it (670 of 4700
    // cycles of a chunk).  Nothing branches: the last chunk's copies of a chunk
    // that is not there read an empty buffer.
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    constexpr int kKeySteps = Regs::kKeys, kSteps = kKeySteps + 3;
    // A thread's or wave's piece of the keys (then queries) may be none.
    auto none = [&](bool is_q) { return !OUT && is_q; };
    auto keys_or_queries = [&](Buf &to, bool is_q, int e) __attribute__((always_inline)) {
        if constexpr (OUT) return is_q ? &to.q[e][0][0] : &to.k[e][0][0];
        else return &to.k[e][0][0];
    };
    uint32_t kq_off[kKeySteps], v_off;
    auto is_query = [&](int k) { return 4 * k + uwave >= 2 * NB; };
    if constexpr (DIRECT) {
#pragma unroll
        for (int k = 0; k < kKeySteps; ++k) {
            const int at = 64 * (4 * k + uwave - (is_query(k) ? 2 * NB : 0)) + lane, row = at / (4 * NB);
            const int n = 8 * ((at % (4 * NB)) ^ key_swz<NB>(row));
            kq_off[k] = n < N ? 2u * ((uint32_t)row * (uint32_t)(is_query(k) ? p.q_ts : p.k_ts) + (uint32_t)n) : 0xffffff00u;
        }
        const int at = 64 * uwave + lane, row = at / 8, n = 8 * ((at % 8) ^ v_swz<T>(row));
        v_off = n < v_cols ? 2u * ((uint32_t)row * (uint32_t)p.v_ts + (uint32_t)n) : 0xffffff00u;
    }
    // The next chunk's rows, and the tokens from it on (none or fewer: no chunk).
    const T *k_next = kbase, *q_next = qbase, *v_next = vbase;
    const char *pack_next = packs;
    int left_next = tokens;
    auto copy = [&](const void *base, uint32_t bytes, uint32_t off, void *to) __attribute__((always_inline)) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(base, bytes), (__attribute__((address_space(3))) void *)to, 16,
                                                 (int)off, 0, 0, 0);
    };
    auto fetch_step = [&](int k, Buf &to) __attribute__((always_inline)) {
        const uint32_t before = (uint32_t)min(left_next, C) - 1u;  // rows before the last
        auto bytes = [&](int64_t ts, int inner) { return left_next > 0 ? 2u * (before * (uint32_t)ts + (uint32_t)inner) : 0u; };
        if (k < kKeySteps) {
            const bool q = is_query(k);
            if (none(q)) return;
            copy(q ? q_next : k_next, bytes(q ? p.q_ts : p.k_ts, N), kq_off[k],
                 keys_or_queries(to, q, 0) + 512 * (4 * k + uwave - (q ? 2 * NB : 0)));
        } else if (k == kKeySteps) {
            copy(v_next, map ? 0u : bytes(p.v_ts, v_cols), v_off, &to.v[0][0] + 512 * uwave);
        } else {
            const int at = 1024 * (4 * (k - kKeySteps - 1) + uwave);
            copy(pack_next, left_next > 0 ? (uint32_t)L::kUsed : 0u, (uint32_t)at + 16u * lane, to.pack + at);
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        k_next += C * p.k_ts;
        q_next += C * p.q_ts;
        v_next += C * p.v_ts;
        pack_next += pack_stride;
        left_next -= C;
    };
    // Through registers: eight elements per piece; rows past the end repeat the last one (their u
    // are 0), columns past N are 0.  A thread's pieces keep their rows and
    // columns, so their addresses only move on by a chunk; they are taken anew
    // for the last one, which may be cut short.
    const T *kq_at[kKeySteps], *v_at;
    const int v_row = tid >> 3, v_col = 8 * (tid & 7);
    auto piece_of = [&](int i, bool &is_q, int &row, int &n) {
        const int at = tid + kThreads * i;
        is_q = at >= 128 * NB;
        const int piece = is_q ? at - 128 * NB : at;
        row = piece / (4 * NB);
        n = 8 * (piece % (4 * NB));
    };
    auto point = [&]() {  // at the next chunk
        const int left = min(left_next, C) - 1;  // the last row
#pragma unroll
        for (int i = 0; i < kKeySteps; ++i) {
            bool is_q;
            int row, n;
            piece_of(i, is_q, row, n);
            const int64_t t = min(row, left);
            kq_at[i] = (is_q ? q_next + t * p.q_ts : k_next + t * p.k_ts) + min(n, N - 8);
        }
        v_at = v_next + (int64_t)min(v_row, left) * p.v_ts + min(v_col, max(v_cols, 8) - 8);
    };
    auto fetch = [&](Regs &r, Buf &to) __attribute__((always_inline)) {
        if (left_next < C) point();
#pragma unroll
        for (int i = 0; i < kKeySteps; ++i) {
#pragma unroll
            for (int j = 0; j < Regs::WORDS; ++j) r.kq[i][j] = load_words(kq_at[i] + j * Regs::VEC);
            bool is_q;
            int row, n;
            piece_of(i, is_q, row, n);
            kq_at[i] += C * (is_q ? p.q_ts : p.k_ts);
        }
#pragma unroll
        for (int j = 0; j < Regs::WORDS; ++j) r.v[j] = load_words(v_at + j * Regs::VEC);
        v_at += C * p.v_ts;
        const char *src = pack_next;
        if constexpr (BUFS == 2) {
            // The other buffer's last reader is behind the last barrier.
#pragma unroll
            for (int i = 0; i < Regs::kPackWords; ++i) {
                const int at = 16 * (kThreads * i + 64 * wave);
                if (at + 1024 <= L::kUsed || at + 16 * lane < L::kUsed) copy16_to_lds(src + at + 16 * lane, to.pack + at);
            }
        } else {
#pragma unroll
            for (int i = 0; i < Regs::kPackWords; ++i)
                r.pack[i] = reinterpret_cast<const u32x4 *>(src)[min(tid + kThreads * i, L::kBytes / 16 - 1)];
        }
    };
    auto place = [&](const Regs &r, Buf &to) {
#pragma unroll
        for (int i = 0; i < kKeySteps; ++i) {
            bool is_q;
            int row, n;
            piece_of(i, is_q, row, n);
            if (n >= N || none(is_q)) continue;
            const int in_plane = row * Buf::kPlane + (n ^ 8 * key_swz<NB>(row));
            if constexpr (NI == 1) {
                *reinterpret_cast<u32x4 *>(keys_or_queries(to, is_q, 0) + in_plane) = r.kq[i][0];
            } else {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = word_f32(r.kq[i][e / 4], e % 4, float());
                bf16x8 t[3];
                split(f, t);
#pragma unroll
                for (int e = 0; e < NI; ++e)
                    *reinterpret_cast<bf16x8 *>(keys_or_queries(to, is_q, e) + in_plane) = t[e];
            }
        }
#pragma unroll
        for (int j = 0; j < Regs::WORDS; ++j)
            *reinterpret_cast<u32x4 *>(&to.v[v_row][(v_col ^ 8 * v_swz<T>(v_row)) + j * Regs::VEC]) =
                map ? u32x4{0u, 0u, 0u, 0u} : r.v[j];
        if constexpr (BUFS == 1)
#pragma unroll
            for (int i = 0; i < Regs::kPackWords; ++i)
                if (tid + kThreads * i < L::kBytes / 16) *reinterpret_cast<u32x4 *>(to.pack + 16 * (tid + kThreads * i)) = r.pack[i];
    };

    // Tile (kb, half) of the state: rows n = 32 kb + 8 g + 4 half + r, column p0 +
    // i16; the two halves' eight rows of a lane are consecutive.
    f32x4 s[NB][2];
    const int64_t s_off = (int64_t)((live ? p0 : 0) + i16) * N + 8 * g, v_state = (int64_t)p.headdim * N;
    auto store_state = [&](const f32x4 (&m)[NB][2], float *to) {
        if (!live) return;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
            if (32 * kb + 8 * g < N) {
                *reinterpret_cast<f32x4 *>(to + s_off + 32 * kb) = m[kb][0];
                *reinterpret_cast<f32x4 *>(to + s_off + 32 * kb + 4) = m[kb][1];
            }
    };
    // Of range r, [range][b,h][P,N]: its final state, later the state that enters
    // range r + 1.
    auto range_state = [&](unsigned r) { return p.range_state + ((int64_t)r * p.batch * p.nheads + bh) * v_state; };
    const float *from = nullptr;
    if (OUT && range > 0) from = range_state(range - 1);
    else if (OUT && p.ranges > 1) from = p.init_state ? p.range_init + bh * v_state : nullptr;
    else if (range == 0 && p.init_state) from = p.init_state + bh * v_state;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
        s[kb][0] = s[kb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (from && 32 * kb + 8 * g < N) {
            s[kb][0] = *reinterpret_cast<const f32x4 *>(from + s_off + 32 * kb);
            s[kb][1] = *reinterpret_cast<const f32x4 *>(from + s_off + 32 * kb + 4);
        }
        if (map)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[kb][i >> 2][i & 3] = 32 * kb + 8 * g + i == p0 + i16 ? 1.0f : 0.0f;
    }
    int at = -1;  // the accepted index within this range, none of its own below 0
    if (OUT && p.state_out) {
        const int64_t j = min(max((int64_t)p.state_out_idx[b], (int64_t)-1), p.seqlen - 1);
        if (j < 0 && range == 0) store_state(s, p.state_out + bh * v_state);
        at = j >= first && j < first + tokens ? (int)(j - first) : -1;
    }

    // K' of a chunk as an operand with rows n of tile (kb, half) and the tokens
    // 4 g + r of both token tiles as the contraction.
    auto keys_t = [&](const Buf &buf, int kb, int half, bf16x8 (&f)[NI]) {
#pragma unroll
        for (int e = 0; e < NI; ++e) {
            // Row r + 16 has the swizzle of row r.
            const int row = 4 * g + (i16 >> 2);
            const bf16 *src = &buf.k[e][row][((32 * kb + 8 * (i16 & 3)) ^ 8 * key_swz<NB>(row)) + 4 * half];
            const i16x4 lo = ds_read_tr16(src), hi = ds_read_tr16(src + 16 * Buf::kPlane);
            typedef short i16x8 __attribute__((ext_vector_type(8)));
            f[e] = __builtin_bit_cast(bf16x8, (i16x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    };

    if (!DIRECT && N < 32 * NB) {  // columns that no piece fills
        for (int i = tid; i < (int)sizeof(Buf) / 16; i += kThreads)
            reinterpret_cast<u32x4 *>(&buf0)[i] = reinterpret_cast<u32x4 *>(&buf1)[i] = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
    }
    Regs regs;
    if constexpr (DIRECT) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) fetch_step(k, buf0);
    } else {
        point();
        fetch(regs, buf0);
        place(regs, buf0);
    }
    advance();
    // Outputs by a buffer over the chunk's rows, which drops those past the end.
    const uint32_t y_row = (uint32_t)(p.nheads * p.headdim * (int)sizeof(T));
    const uint32_t y_off = (uint32_t)i16 * y_row + (uint32_t)(((int)h * p.headdim + p0 + 4 * g) * (int)sizeof(T));
    wait_vmcnt<0>();
    __syncthreads();
    char *y_at = reinterpret_cast<char *>(p.y) + ((int64_t)b * p.seqlen + first) * (int64_t)y_row;
    bf16x4 minus_one;  // -1 times the identity
#pragma unroll
    for (int r = 0; r < 4; ++r) minus_one[r] = i16 == 4 * g + r ? (bf16)-1.0f : (bf16)0.0f;
    // The chunk whose first token is `t` from `buf`, while the next one comes into
    // `other`.
    auto chunk = [&](int t, const Buf &buf, Buf &other) __attribute__((always_inline)) {
        const bool more = left_next > 0;
        if (!DIRECT && more) fetch(regs, other);
        // A wave without rows issues its copies at once.
        auto fetch_some = [&](int from, int to) {
            if constexpr (DIRECT)
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
                    if (k >= from && k < to) fetch_step(k, other);
        };
        if (!live) fetch_some(0, kSteps);
        f32x4 qs[2] = {};  // S q, then y
        if (live) {
            const float *tab = reinterpret_cast<const float *>(buf.pack + L::kTab);
            // What a term leaves of the state or of the updates is a product of the
            // matrix cores too: the tile minus the unit matrix times the term, exact, in
            // the place of two vector instructions per value, which such a wave is bound
            // by (7% of the time of 16384 tokens of 32 heads in one range with the state's,
            // 2% of 2 x 4096 tokens with the updates').  The state's terms are taken
            // a step ahead, so that nothing waits for them; where the registers do not
            // hold that, or a lone wave per SIMD would wait, they are subtracted.
            constexpr bool AHEAD = WAVES == 2 && (NB <= 4 || DIRECT);
            auto split_tiles = [&](const f32x4 (&v)[2], auto &to) __attribute__((always_inline)) {
                constexpr int TERMS = sizeof(to) / sizeof(bf16x8);
                f32x4 left[2] = {v[0], v[1]};
#pragma unroll
                for (int e = 0; e < TERMS; ++e) {
                    float f[8];
                    bf16x8 t[1];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = left[i >> 2][i & 3];
                    split(f, t);
                    to[e] = t[0];
                    if (e + 1 < TERMS)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            left[half] = mfma(minus_one, half ? bf16x4{t[0][4], t[0][5], t[0][6], t[0][7]}
                                                              : bf16x4{t[0][0], t[0][1], t[0][2], t[0][3]}, left[half]);
                }
            };
            auto split_values = [&](const float (&v)[8], auto &to) __attribute__((always_inline)) {
                if constexpr (AHEAD) {
                    const f32x4 tiles[2] = {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
                    split_tiles(tiles, to);
                } else {
                    split(v, to);
                }
            };
            // The order of what follows is written out, since with two waves per
            // SIMD at most a read of LDS right before its use costs its latency:
            // every operand is read one step ahead (a scheduling barrier keeps
            // it there), and the products that only the outputs need (S q) stand
            // where the chain S k -> X -> U waits for the matrix cores.
            auto rows_of = [&](const bf16 (&plane)[NI][C][Buf::kPlane], int kb, bf16x8 (&f)[2][NI]) {
#pragma unroll
                for (int I = 0; I < 2; ++I)
#pragma unroll
                    for (int e = 0; e < NI; ++e)
                        f[I][e] = *reinterpret_cast<const bf16x8 *>(
                            &plane[e][16 * I + i16][(32 * kb + 8 * g) ^ 8 * key_swz<NB>(i16)]);
            };
            // S k (rows: tokens); the terms of S are kept for S q (rows: p).
            f32x4 ks[2] = {};
            bf16x8 sf[NB][3], kf[2][2][NI], qf[2][2][NI];
            auto split_state = [&](int kb) { split_tiles(s[kb], sf[kb]); };
            rows_of(buf.k, 0, kf[0]);
            if constexpr (AHEAD) split_state(0);
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                if (kb + 1 < NB) rows_of(buf.k, kb + 1, kf[(kb + 1) & 1]);
                else if constexpr (OUT) rows_of(buf.q, 0, qf[0]);
                if (kb < kKeySteps) fetch_some(kb, kb + 1);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (AHEAD) {
                    if (kb + 1 < NB) split_state(kb + 1);
#pragma unroll
                    for (int I = 0; I < 2; ++I) mma_terms<NI, 3>(kf[kb & 1][I], sf[kb], ks[I]);
                } else {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = s[kb][i >> 2][i & 3];
                    split(f, sf[kb]);
#pragma unroll
                    for (int I = 0; I < 2; ++I) mma_terms<NI, 3>(kf[kb & 1][I], sf[kb], ks[I]);
                }
            }
            auto s_q = [&](int kb) {
                if constexpr (OUT)
                    if (kb + 1 < NB) rows_of(buf.q, kb + 1, qf[(kb + 1) & 1]);
                fetch_some(kKeySteps + (kb == 0 ? 0 : kb + 1), kb + 1 == NB ? kSteps : kKeySteps + kb + 2);
                __builtin_amdgcn_sched_barrier(0);
                if (OUT)
#pragma unroll
                    for (int I = 0; I < 2; ++I) mma_terms<3, NI>(sf[kb], qf[kb & 1][I], qs[I]);
            };
            // X = v - a S k.
            f32x4 av[2];
            float x[8];
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                av[I] = *reinterpret_cast<const f32x4 *>(tab + L::kA + 16 * I + 4 * g);
                if constexpr (sizeof(T) == 2) {
                    const int row = 16 * I + 4 * g + (i16 >> 2), col = 16 * wave + 4 * (i16 & 3);
                    const i16x4 t = ds_read_tr16(&buf.v[row][col ^ 8 * v_swz<T>(row)]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[4 * I + r] = __builtin_bit_cast(float, (uint32_t)(uint16_t)t[r] << 16);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[4 * I + r] = buf.v[16 * I + 4 * g + r][16 * wave + i16];
                }
            }
            s_q(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(-av[i >> 2][i & 3], ks[i >> 2][i & 3], x[i]);
            // U = Tb X.
            [[maybe_unused]] f32x4 tt[3];
            [[maybe_unused]] bf16x4 t0[3];
            [[maybe_unused]] bf16x8 t1[3];
            auto tables = [&](int off0, int off1, f32x4 (&tiles)[3], bf16x4 (&half)[3], bf16x8 (&both)[3]) {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if constexpr (L::kTerms) {
                        half[e] = *reinterpret_cast<const bf16x4 *>(buf.pack + off0 + (e * 64 + lane) * 8);
                        both[e] = *reinterpret_cast<const bf16x8 *>(buf.pack + off1 + (e * 64 + lane) * 16);
                    } else {
                        tiles[e] = *reinterpret_cast<const f32x4 *>(buf.pack + off0 + (e * 64 + lane) * 16);
                    }
            };
            tables(L::kT0, L::kT1, tt, t0, t1);
            if (NB > 1) s_q(1);
            else __builtin_amdgcn_sched_barrier(0);
            f32x4 u[2] = {}, dv[2];
            if constexpr (L::kTerms) {
                bf16x4 x0[3];
                bf16x8 xf[3];
                split(x, xf);  // the chain waits for this one
#pragma unroll
                for (int e = 0; e < 3; ++e) x0[e] = bf16x4{xf[e][0], xf[e][1], xf[e][2], xf[e][3]};
                mma_terms<3, 3>(t0, x0, u[0]);
                mma_terms<3, 3>(t1, xf, u[1]);
            } else {
                const f32x4 xt[2] = {{x[0], x[1], x[2], x[3]}, {x[4], x[5], x[6], x[7]}};
                u[0] = mma_f32_16(tt[0], xt[0], u[0]);
                u[1] = mma_f32_16(tt[1], xt[0], u[1]);
                u[1] = mma_f32_16(tt[2], xt[1], u[1]);
            }
#pragma unroll
            for (int kb = 2; kb < NB; ++kb) s_q(kb);
            [[maybe_unused]] f32x4 pm[3];
            [[maybe_unused]] bf16x4 pm0[3];
            [[maybe_unused]] bf16x8 pm1[3];
            tables(L::kP0, L::kP1, pm, pm0, pm1);
            float cv[2];
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                cv[I] = tab[L::kC + 16 * I + i16];
                dv[I] = *reinterpret_cast<const f32x4 *>(tab + L::kD + 16 * I + 4 * g);
            }
            const float end = tab[L::kEnd];
            __builtin_amdgcn_sched_barrier(0);
            if (at >= t && at - t < C) {  // the state after the accepted index
                const float *wt = p.at_tables + (int64_t)bh * kAtFloats;
                const float e = wt[C];
                float uv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) uv[i] = u[i >> 2][i & 3] * wt[16 * (i >> 2) + 4 * g + (i & 3)];
                bf16x8 uf[3];
                split_values(uv, uf);
                f32x4 m[NB][2];
#pragma unroll
                for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        bf16x8 kt[NI];
                        keys_t(buf, kb, half, kt);
#pragma unroll
                        for (int r = 0; r < 4; ++r) m[kb][half][r] = s[kb][half][r] * e;
                        mma_terms<NI, 3>(kt, uf, m[kb][half]);
                    }
                store_state(m, p.state_out + bh * v_state);
            }
            // y: rows p = p0 + 4 g + r, column: token 16 I + i16.
            if constexpr (OUT) {
#pragma unroll
                for (int I = 0; I < 2; ++I)
#pragma unroll
                    for (int r = 0; r < 4; ++r) qs[I][r] *= cv[I];
                if constexpr (L::kTerms) {
                    const float uv[8] = {u[0][0], u[0][1], u[0][2], u[0][3], u[1][0], u[1][1], u[1][2], u[1][3]};
                    bf16x8 uf[3];
                    bf16x4 u0[3];
                    split_values(uv, uf);
#pragma unroll
                    for (int e = 0; e < 3; ++e) u0[e] = bf16x4{uf[e][0], uf[e][1], uf[e][2], uf[e][3]};
                    mma_terms<3, 3>(u0, pm0, qs[0]);
                    mma_terms<3, 3>(uf, pm1, qs[1]);
                } else {
                    qs[0] = mma_f32_16(u[0], pm[0], qs[0]);
                    qs[1] = mma_f32_16(u[0], pm[1], qs[1]);
                    qs[1] = mma_f32_16(u[1], pm[2], qs[1]);
                }
            }
            // The state after the chunk.
            {
                bf16x8 kt[2][NI];
                keys_t(buf, 0, 0, kt[0]);
                keys_t(buf, 0, 1, kt[1]);
                __builtin_amdgcn_sched_barrier(0);
                float uv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) uv[i] = u[i >> 2][i & 3] * dv[i >> 2][i & 3];
                bf16x8 uf[3];
                split_values(uv, uf);
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) {
                    bf16x8 next[2][NI];
                    if (kb + 1 < NB) {
                        keys_t(buf, kb + 1, 0, next[0]);
                        keys_t(buf, kb + 1, 1, next[1]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[kb][half][r] *= end;
                        mma_terms<NI, 3>(kt[half], uf, s[kb][half]);
                    }
                    if (kb + 1 < NB)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
#pragma unroll
                            for (int e = 0; e < NI; ++e) kt[half][e] = next[half][e];
                }
            }
        }
        // The loads of the next chunk are waited for before the outputs are
        // stored: the counter would make the wait include the stores.
        if (BUFS == 2) wait_vmcnt<0>();  // among them the copies into the other buffer
        else __syncthreads();            // the only buffer is read no more
        if (!DIRECT && more) place(regs, other);
        __builtin_amdgcn_sched_barrier(0);
        if (OUT && live)
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                if constexpr (DIRECT) {
                    const __amdgpu_buffer_rsrc_t yr = buffer_rsrc(y_at, (uint32_t)min(tokens - t, C) * y_row);
                    const bf16x4 o = {(bf16)qs[I][0], (bf16)qs[I][1], (bf16)qs[I][2], (bf16)qs[I][3]};
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), yr, (int)(y_off + 16u * I * y_row), 0, 0);
                } else if (16 * I + i16 < tokens - t) {
                    T *to = reinterpret_cast<T *>(y_at + (int64_t)(16 * I + i16) * y_row) + (int64_t)h * p.headdim + p0 + 4 * g;
                    if constexpr (sizeof(T) == 2) {
                        const bf16x4 o = {(bf16)qs[I][0], (bf16)qs[I][1], (bf16)qs[I][2], (bf16)qs[I][3]};
                        *reinterpret_cast<u32x2_at2 *>(to) = __builtin_bit_cast(u32x2, o);
                    } else {
                        store_words(to, __builtin_bit_cast(u32x4, qs[I]));
                    }
                }
            }
        y_at += (int64_t)C * y_row;
        advance();
        __syncthreads();
    };
    if constexpr (BUFS == 2) {
        for (int left = tokens; left > 0; left -= 2 * C) {
            chunk(tokens - left, buf0, buf1);
            if (left > C) chunk(tokens - left + C, buf1, buf0);
        }
    } else {
        for (int left = tokens; left > 0; left -= C) chunk(tokens - left, buf0, buf0);
    }
    if constexpr (OUT) {
        if (p.final_state && range + 1 == ranges) store_state(s, p.final_state + bh * v_state);
    } else {
        if (map) store_state(s, p.range_map + ((int64_t)(range - 1) * p.batch * p.nheads + bh) * N * N);
        else store_state(s, range_state(range));
    }
}

// Between the passes: the states that enter the ranges, S_{r+1} = S_r M_r + D_r
// one after the other, in place of the D_r.  A workgroup per (b, h, 16 rows), a
// wave per 16 columns, fp32 products; S_r passes through LDS.  The ranges follow
// one another, so latency sets the time: a range's whole map is loaded while the
// one before is multiplied (62 -> 16 us for 8 ranges of 32 heads, N and P 128;
// loads inside the products' loop wait for each step).  It also sets init_state
// aside, which the last range may overwrite (in-place calls) before the first one
// starts.
constexpr int kJoinRow = 256 + 4;
template <int NT>  // N / 16
__global__ __launch_bounds__(64 * NT) void delta_join(DeltaParams p) {
    __shared__ __attribute__((aligned(16))) float held[16][kJoinRow];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i16 = lane & 15, g = lane >> 4;
    constexpr int N = 16 * NT;
    // Tiles of a head lie nheads apart, so they share an L2 where that is a multiple of 8.
    const unsigned heads = (unsigned)(p.batch * p.nheads), tile = blockIdx.x / heads, bh = blockIdx.x - tile * heads;
    const int64_t BH = heads, v_state = (int64_t)p.headdim * N, mine = bh * v_state + (int64_t)tile * 16 * N;
    if (p.init_state)
        for (int i = 4 * tid; i < 16 * N; i += 4 * (int)blockDim.x)
            *reinterpret_cast<f32x4 *>(p.range_init + mine + i) = *reinterpret_cast<const f32x4 *>(p.init_state + mine + i);
    for (int i = 4 * tid; i < 16 * N; i += 4 * (int)blockDim.x)
        *reinterpret_cast<f32x4 *>(&held[i / N][i % N]) = *reinterpret_cast<const f32x4 *>(p.range_state + mine + i);
    const int n = 16 * wave + i16;  // this lane's column, rows 4 g + r
    f32x4 map[NT], acc;             // a range's map and state, read a range ahead
    const unsigned at = 4 * g * N + n;
    auto fetch = [&](int r) {
        const float *m = p.range_map + ((int64_t)(r - 1) * BH + bh) * N * N;
        const float *d = p.range_state + (int64_t)r * BH * v_state + mine;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) map[j][k] = (m + (16 * j + k) * N)[at];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = (d + k * N)[at];
    };
    if (p.ranges > 2) fetch(1);
    __syncthreads();
    for (int r = 1; r + 1 < p.ranges; ++r) {
        f32x4 sum = acc;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            sum = mma_f32_16(*reinterpret_cast<const f32x4 *>(&held[i16][16 * j + 4 * g]), map[j], sum);
        if (r + 2 < p.ranges) fetch(r + 1);
        __syncthreads();
        float *d = p.range_state + (int64_t)r * BH * v_state + mine;
#pragma unroll
        for (int k = 0; k < 4; ++k) held[4 * g + k][n] = (d + k * N)[at] = sum[k];
        __syncthreads();
    }
}

// The LDS buffers of a workgroup, and the waves per SIMD that LDS and the size of
// the state leave.  One buffer where two workgroups fit a unit with one each but
// not with two, and the registers hold what then passes through them: fp32, N 64
// and 96, 64 and 32 heads of 8 x 1024 and 8 x 512 tokens 191 -> 170 and 118 -> 101
// us (N 128, which spills: 137 -> 168).
constexpr int kLds = 160 * 1024;
template <typename T, int NB, bool OUT>
constexpr int buffers() {
    static_assert(sizeof(Buffer<T, NB, OUT>) <= kLds, "LDS");
    constexpr size_t bytes = sizeof(Buffer<T, NB, OUT>);
    if (NB <= 3 && 2 * bytes <= kLds && 4 * bytes > kLds) return 1;
    return 2 * bytes <= kLds ? 2 : 1;
}
template <typename T, int NB, bool OUT>
constexpr int waves_per_simd() {
    return 2 * buffers<T, NB, OUT>() * sizeof(Buffer<T, NB, OUT>) <= kLds && NB <= 5 ? 2 : 1;
}

template <typename T, int NB>
hipError_t launch(const DeltaParams &given, hipStream_t stream) {
    // As many heads per wave of the preparation as share their keys while that
    // leaves two waves per SIMD (their rows are loaded and multiplied once: 62 ->
    // 40 us for 512 chunks of 32 heads in 8 groups).
    DeltaParams p = given;
    p.prepare_heads = 1;
    for (int d = 2; d <= p.heads_per_group && d <= 8; ++d)
        if (p.heads_per_group % d == 0 && p.batch * p.nchunks * (p.nheads / d) >= 2 * 1024) p.prepare_heads = d;
    const int64_t waves = p.batch * p.nchunks * (p.nheads / p.prepare_heads);
    delta_prepare<T, NB><<<(unsigned)((waves + kThreads / 64 - 1) / (kThreads / 64)), kThreads, 0, stream>>>(p);
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    const int64_t v_slices = (p.headdim + kSlice - 1) / kSlice, n_slices = (p.dstate + kSlice - 1) / kSlice;
    const int64_t heads = p.batch * p.nheads;
    auto passes = [&](auto direct) {
        constexpr bool D = decltype(direct)::value;
        if (p.ranges > 1) {
            delta_chunks<T, NB, buffers<T, NB, false>(), waves_per_simd<T, NB, false>(), D, false>
                <<<(unsigned)(heads * (p.ranges - 1) * (v_slices + n_slices)), kThreads, 0, stream>>>(p);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const unsigned tiles = (unsigned)(heads * (p.headdim / 16)), threads = 4 * p.dstate;
            if (p.dstate % 32) delta_join<2 * NB - 1><<<tiles, threads, 0, stream>>>(p);
            else delta_join<2 * NB><<<tiles, threads, 0, stream>>>(p);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        delta_chunks<T, NB, buffers<T, NB, true>(), waves_per_simd<T, NB, true>(), D, true>
            <<<(unsigned)(heads * p.ranges * v_slices), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    };
    if constexpr (sizeof(T) == 2) {
        // Direct copies need rows of 16-byte alignment and 32-bit offsets within a
        // chunk (the last byte below 2^31, so that the mark of no element is out).
        auto fits = [&](const void *base, int64_t bs, int64_t ts, int64_t inner) {
            return (uintptr_t)base % 16 == 0 && bs % 8 == 0 && ts % 8 == 0 && C * ts + inner < ((int64_t)1 << 30);
        };
        const int64_t y_bytes = (int64_t)C * p.nheads * p.headdim * 2;
        if (fits(p.q, p.q_bs, p.q_ts, 256) && fits(p.k, p.k_bs, p.k_ts, 256) && fits(p.v, p.v_bs, p.v_ts, 256) &&
            (uintptr_t)p.y % 16 == 0 && y_bytes < ((int64_t)1 << 31))
            return passes(std::true_type{});
    }
    return passes(std::false_type{});
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

// Few heads leave most of the GPU idle while their chunks are walked one after
// the other, so a long sequence is cut into ranges of chunks that run side by
// side, twice (see delta_chunks), with a join between.  In units of a chunk's
// time with one workgroup per compute unit, a pass over ranges of L chunks takes
// L, (1 + 3 k) / 4 L where k workgroups share a unit, and as often that as the GPU has
// to be filled; the first pass computes no outputs (0.65), and its workgroups are
// more (the maps' rows); the launches and the join add about 2 + r.  Measured,
// 16384 tokens of 32 heads (N and P 128, bf16) in 1, 2, 3, 4, 5, 7, 8, 10 and 16
// ranges: 876, 775, 541, 492, 506, 457, 460, 509 and 494 us; 1021 tokens of 30
// heads (N 96, P 80, fp32) in 1, 2, 3, 4, 5 and 6: 107, 97, 77, 72, 76 and 81 us;
// 32768 tokens of 8 heads in 1, 4, 8 and 16: 1696, 769, 424 and 298 us; 2 x 4096
// tokens of 32 heads in 1, 2, 3 and 4: 235, 213, 223 and 214 us.  Of 35 shapes (N 32
// to 256, 8 to 32 heads, 2048 to 8192 tokens) the choice was within 7% of the best of
// 12 numbers of ranges at 27, and 23% off at worst (2048 tokens of 16 heads, P 64, N
// 128, fp32: 117 us in four, 95 in twelve).
void delta_ranges(DeltaParams &p, Elem e) {
    p.ranges = 1;
    p.range_chunks = p.nchunks;
    if (p.nchunks < 2) return;
    const double heads = (double)p.batch * p.nheads;
    const int v_slices = (p.headdim + kSlice - 1) / kSlice, n_slices = (p.dstate + kSlice - 1) / kSlice;
    // Workgroups that fit a compute unit in either pass, by ceil(N / 32): LDS and the
    // registers of the compiled instances (bf16: of direct copies; rows that pass
    // through registers leave up to two fewer, with which the choice is no better).
    static constexpr int kFit[2][2][8] = {{{3, 2, 2, 1, 1, 1, 1, 1}, {2, 2, 2, 1, 1, 1, 1, 1}},   // fp32
                                          {{5, 5, 4, 4, 3, 2, 2, 2}, {4, 4, 3, 2, 2, 1, 1, 1}}};  // bf16
    const int nb = (p.dstate + 31) / 32 - 1;
    const double fit_first = kFit[e == Elem::BF16][0][nb], fit_second = kFit[e == Elem::BF16][1][nb];
    auto rounds = [](double wgs, double fit) {
        const double each = ceil(wgs / 256.0), whole = floor(each / fit), rest = each - whole * fit;
        return whole * (0.25 + 0.75 * fit) + (rest > 0.0 ? 0.25 + 0.75 * rest : 0.0);
    };
    double best = 0.9 * (double)p.nchunks * rounds(heads * v_slices, fit_second);
    for (int r = 2; r <= 16; ++r) {
        const int64_t len = (p.nchunks + r - 1) / r;
        if ((p.nchunks + len - 1) / len != r) continue;  // fewer ranges of this length
        const double first = heads * (v_slices + (r - 2) * (v_slices + n_slices)), second = heads * v_slices * r;
        const double cost = (double)len * (0.65 * rounds(first, fit_first) + rounds(second, fit_second)) + 2.0 + r;
        if (cost < best) {
            best = cost;
            p.ranges = r;
            p.range_chunks = len;
        }
    }
}

size_t delta_pack_bytes(Elem e) { return e == Elem::BF16 ? Pack32<bf16>::kBytes : Pack32<float>::kBytes; }
size_t delta_at_bytes() { return kAtFloats * sizeof(float); }

hipError_t launch_delta_chunks(const DeltaParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
