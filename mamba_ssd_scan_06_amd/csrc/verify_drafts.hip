// Verification of drafted tokens: per sequence the first draft i with
// u_i q_i(tok_i) >= p_i(tok_i), then a token from the residual
// r = max(p_n - q_n, 0) (p_m when every draft is accepted) by inverse CDF.
//
// Everything that decides is fp64: u q is exact there (24-bit factors), and
// sums of fp32 values keep 29 spare bits, so that the order in which a row is
// summed moves a border between two tokens by 1e-16 of the row's mass only.
// The order is fixed, so equal inputs give equal tokens.
//
// Only the K tested probabilities and one row of p and q are needed.  A row is
// summed in segments; the prefix over their sums finds the segment that holds
// the cut, which is read again (from cache) with a few adjacent elements per
// thread.  With many sequences a workgroup of 16 waves takes a whole row, its
// waves' pieces being the segments; with few, a first launch sums the segments
// of all rows on the whole GPU and a workgroup per row picks the token.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSumThreads = 256;
constexpr int kMaxSegments = 64;

// A probability's mass: NaN and negative values count as none.
__device__ __forceinline__ double mass(double v) { return __builtin_fmax(v, 0.0); }

// Inclusive prefix sums over a wave's lanes.
__device__ __forceinline__ double lane_prefix(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const double o = __shfl_up(v, k);
        if (lane >= k) v += o;
    }
    return v;
}

// What a sequence's drafts leave: the row to draw from.
template <typename T>
struct Residual {
    const T *p, *q;   // rows of the target and the draft (null without)
    int64_t zeroed;   // token whose mass is taken away, or -1
    bool drawn;       // a draft was rejected: r is the residual, not p itself

    __device__ __forceinline__ double at(int64_t v) const {
        const double pv = (double)to_f32(p[v]);
        if (q) return mass(pv - (double)to_f32(q[v]));
        return v == zeroed ? 0.0 : mass(pv);
    }
    // Sum over [lo, hi) by the 64 lanes of a wave, each adding 16 bytes of
    // elements at a time; the same in every lane.
    __device__ __forceinline__ double wave_sum(int64_t lo, int64_t hi) const {
        constexpr int VEC = 16 / sizeof(T);
        const int lane = threadIdx.x & 63;
        double s = 0.0;
        int64_t v = lo + lane * VEC;
        auto add = [&](const Pack<T, VEC> &pv, const Pack<T, VEC> &qv, int64_t from) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const double d = (double)to_f32(pv.v[i]);
                s += q ? mass(d - (double)to_f32(qv.v[i])) : from + i == zeroed ? 0.0 : mass(d);
            }
        };
        constexpr int STEP = 64 * VEC, U = 4;
        for (; v + (U - 1) * STEP + VEC <= hi; v += U * STEP) {
            Pack<T, VEC> pv[U], qv[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                pv[k] = *reinterpret_cast<const Pack<T, VEC> *>(p + v + k * STEP);
                if (q) qv[k] = *reinterpret_cast<const Pack<T, VEC> *>(q + v + k * STEP);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) add(pv[k], qv[k], v + k * STEP);
        }
        for (; v < hi; v += STEP) {
            if (v + VEC <= hi) {
                Pack<T, VEC> pv = *reinterpret_cast<const Pack<T, VEC> *>(p + v), qv = {};
                if (q) qv = *reinterpret_cast<const Pack<T, VEC> *>(q + v);
                add(pv, qv, v);
            } else {
                for (int64_t k = v; k < hi; ++k) s += at(k);
            }
        }
        for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
        return s;
    }
};

__device__ __forceinline__ int drafts_of(const VerifyParams &p, int64_t b) {
    const int m = p.lens ? p.lens[b] : p.drafts;
    return m < 0 ? 0 : (m > p.drafts ? p.drafts : m);
}

// The number of accepted drafts of sequence b, by all threads of a workgroup;
// *first is LDS.
template <typename T>
__device__ __forceinline__ int accepted_drafts(const VerifyParams &p, int64_t b, int m, int *first) {
    if (threadIdx.x == 0) *first = m;
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
        const int32_t v = p.tok[b * p.drafts + i];
        bool ok = v >= 0 && v < p.vocab;
        if (ok) {
            const double q =
                p.draft ? (double)to_f32(reinterpret_cast<const T *>(p.draft)[b * p.d_bs + i * p.d_rs + v]) : 1.0;
            ok = (double)p.u[b * (p.drafts + 1) + i] * q <
                 (double)to_f32(reinterpret_cast<const T *>(p.target)[b * p.t_bs + i * p.t_rs + v]);
        }
        if (!ok) atomicMin(first, i);
    }
    __syncthreads();
    return *first;
}

template <typename T>
__device__ __forceinline__ Residual<T> residual_of(const VerifyParams &p, int64_t b, int n, int m) {
    Residual<T> r;
    r.p = reinterpret_cast<const T *>(p.target) + b * p.t_bs + n * p.t_rs;
    r.drawn = n < m;
    r.q = r.drawn && p.draft ? reinterpret_cast<const T *>(p.draft) + b * p.d_bs + n * p.d_rs : nullptr;
    r.zeroed = r.drawn && !p.draft ? (int64_t)p.tok[b * p.drafts + n] : -1;
    return r;
}

// First launch of a split call: n_accepted and the segments' sums.
template <typename T>
__global__ __launch_bounds__(kSumThreads) void verify_sums_kernel(VerifyParams p) {
    __shared__ int first;
    __shared__ double part[kSumThreads / 64];
    const int64_t b = blockIdx.y;
    const int m = drafts_of(p, b), n = accepted_drafts<T>(p, b, m, &first);
    const Residual<T> r = residual_of<T>(p, b, n, m);
    const int64_t lo = blockIdx.x * p.segment, hi = min(lo + p.segment, p.vocab);
    constexpr int NW = kSumThreads / 64;
    const int64_t per = (hi - lo + NW - 1) / NW;
    const int w = threadIdx.x >> 6;
    const double s = r.wave_sum(min(lo + w * per, hi), min(lo + (w + 1) * per, hi));
    if ((threadIdx.x & 63) == 0) part[w] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int k = 0; k < NW; ++k) sum += part[k];
        p.sums[b * p.segments + blockIdx.x] = sum;
        if (blockIdx.x == 0) p.n_accepted[b] = n;
    }
}

// The rest, one workgroup per sequence.
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyParams p) {
    __shared__ double sums[kMaxSegments], wave_sums[kWaves];
    __shared__ int first, found, last_mass;
    const int64_t b = blockIdx.x, V = p.vocab;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, K = p.drafts;
    const int m = drafts_of(p, b);
    int n;
    if (p.segments > 1) {
        n = p.n_accepted[b];
    } else {
        n = accepted_drafts<T>(p, b, m, &first);
        if (tid == 0) p.n_accepted[b] = n;
    }
    Residual<T> r = residual_of<T>(p, b, n, m);
    int segments = p.segments;
    int64_t segment = p.segment;
    if (segments > 1) {
        if (tid < segments) sums[tid] = p.sums[b * segments + tid];
        __syncthreads();
    }
    double total = 0.0, own = 0.0, upto = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        if (p.segments == 1 || pass == 1) {
            segments = kWaves;
            segment = (V + kWaves - 1) / kWaves;
            const double s = r.wave_sum(min(wave * segment, V), min((wave + 1) * segment, V));
            if (lane == 0) sums[wave] = s;
            __syncthreads();
        }
        // Every wave forms the same prefix over the segments, one per lane.
        own = lane < segments ? sums[lane] : 0.0;
        upto = lane_prefix(own);
        total = __shfl(upto, 63);
        if (total > 0.0 || !r.drawn) break;
        // Rounding left the residual without mass: p_n takes its place.
        r.drawn = false;
        r.q = nullptr;
        r.zeroed = -1;
        __syncthreads();
    }
    const double cut = (double)p.u[b * (K + 1) + K] * total;
    // The segment with the cut: the first whose end passes it, or the last
    // with mass (a uniform outside [0,1), rounding).
    const uint64_t some = __ballot(own > 0.0), past = __ballot(own > 0.0 && upto > cut);
    const int seg = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
    double before = seg > 0 ? __shfl(upto, seg - 1) : 0.0;
    int next = (int)(V - 1);  // a row without mass
    if (seg >= 0) {
        if (tid == 0) {
            found = 0x7fffffff;
            last_mass = -1;
        }
        const int64_t lo = seg * segment, hi = min(lo + segment, V), per = (hi - lo + kThreads - 1) / kThreads;
        const int64_t a = min(lo + tid * per, hi), e = min(a + per, hi);
        double s = 0.0;
#pragma unroll 4
        for (int64_t v = a; v < e; ++v) s += r.at(v);
        const double pre = lane_prefix(s);
        if (lane == 63) wave_sums[wave] = pre;
        __syncthreads();
        {
            const double ends = lane_prefix(lane < kWaves ? wave_sums[lane] : 0.0);
            if (wave > 0) before += __shfl(ends, wave - 1);
        }
        if (s > 0.0) {
            // This thread's elements, from the sum before them.
            double at = before + (pre - s);
            int last = -1;
            for (int64_t v = a; v < e; ++v) {
                const double x = r.at(v);
                if (x > 0.0) last = (int)v;
                at += x;
                if (x > 0.0 && at > cut) {
                    atomicMin(&found, (int)v);
                    break;
                }
            }
            atomicMax(&last_mass, last);
        }
        __syncthreads();
        next = found != 0x7fffffff ? found : last_mass;
    }
    if (tid == 0) p.next_token[b] = next;
    if (p.tokens)
        for (int i = tid; i <= K; i += kThreads)
            p.tokens[b * (K + 1) + i] = i < n ? p.tok[b * K + i] : i == n ? next : -1;
}

template <typename T>
hipError_t run(const VerifyParams &p, hipStream_t stream) {
    if (p.segments > 1) {
        verify_sums_kernel<T><<<dim3(p.segments, (unsigned)p.batch), kSumThreads, 0, stream>>>(p);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
    }
    verify_pick_kernel<T><<<(unsigned)p.batch, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

void verify_segments(VerifyParams &p) {
    // Split while the rows alone leave compute units idle and a segment keeps
    // at least 4096 elements (16 per thread of its workgroup).
    const int64_t want = std::min<int64_t>({kMaxSegments, 256 / std::max<int64_t>(p.batch, 1), p.vocab / 4096});
    p.segments = want >= 4 ? (int)want : 1;
    p.segment = (p.vocab + p.segments - 1) / p.segments;
}

hipError_t launch_verify_drafts(const VerifyParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
