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
// thread.  A workgroup of eight waves takes a whole row, its waves' pieces
// being the segments; where rows are few and long, a first launch sums the
// segments of all rows on the whole GPU and a workgroup per row picks the
// token (verify_segments).  What is left is a chain of latencies: the tested
// probabilities 1 us, a round of a row's loads 1.25 us each (7.8 us of 15.7
// for 256 rows of 50277), two barriers and the segment again 2 us.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kSumThreads = 256;
constexpr int kMaxSegments = 64;  // one per lane
constexpr int kEach = 8;          // elements per thread when a segment is read again

// A probability as it counts: NaN and negative values as 0.
__device__ __forceinline__ float clean(float v) { return __builtin_amdgcn_fmed3f(v, 0.0f, __builtin_inff()); }
// max(p - q, 0) of a cleaned p and any q as p minus the median of p, q and 0
// (min(p, q) for q >= 0; 0 for a negative or NaN q).  Two fp32 values differ
// by an fp64 one exactly, or to 2^-53 of it.
__device__ __forceinline__ double rest(float p, float q) {
    return (double)p - (double)__builtin_amdgcn_fmed3f(p, q, 0.0f);
}

// v plus the value a DPP control moves here (0 where it moves none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double plus_moved(double v) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    const i32x2 x = __builtin_bit_cast(i32x2, v);
    const int lo = __builtin_amdgcn_update_dpp(0, x[0], CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, x[1], CTRL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(double, i32x2{lo, hi});
}
// Inclusive prefix sums over a wave's 64 lanes: shifts within rows of 16, then
// each row's last lane into the rows after it.
__device__ __forceinline__ double lane_prefix(double v) {
    v = plus_moved<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v = plus_moved<0x112, 0xf>(v);
    v = plus_moved<0x114, 0xf>(v);
    v = plus_moved<0x118, 0xf>(v);
    v = plus_moved<0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
    return plus_moved<0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
}
// Lane `lane`'s value, the same for the whole wave.
__device__ __forceinline__ double lane_value(double v, int lane) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    const i32x2 x = __builtin_bit_cast(i32x2, v);
    return __builtin_bit_cast(double, i32x2{__builtin_amdgcn_readlane(x[0], lane), __builtin_amdgcn_readlane(x[1], lane)});
}

// What a sequence's drafts leave: the row to draw from.
template <typename T>
struct Residual {
    const T *p, *q;   // rows of the target and the draft (null without)
    int64_t zeroed;   // token whose mass is taken away, or -1
    bool drawn;       // a draft was rejected: r is the residual, not p itself

    __device__ __forceinline__ double at(int64_t v) const {
        const float f = v == zeroed ? 0.0f : clean(to_f32(p[v]));
        return q ? rest(f, to_f32(q[v])) : (double)f;
    }
    // x[i] = at(v + i); loads first, then their uses.  Beyond `end` x is any value.
    __device__ __forceinline__ void read(int64_t v, int64_t end, double (&x)[kEach]) const {
        constexpr int VEC = 16 / sizeof(T), W = kEach / VEC;
        if (end < kEach) {
            for (int i = 0; i < kEach; ++i) x[i] = at(min(v + i, end - 1));
            return;
        }
        u32x4 pv[W], qv[W];
#pragma unroll
        for (int k = 0; k < W; ++k) pv[k] = load_words(p + v + k * VEC);
        if (q) {
#pragma unroll
            for (int k = 0; k < W; ++k) qv[k] = load_words(q + v + k * VEC);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                x[i] = rest(clean(word_f32(pv[i / VEC], i % VEC, T())), word_f32(qv[i / VEC], i % VEC, T()));
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                x[i] = v + i == zeroed ? 0.0 : (double)clean(word_f32(pv[i / VEC], i % VEC, T()));
        }
    }
    // Sum over [lo, hi) by the 64 lanes of a wave, the same in every lane.
    __device__ __forceinline__ double wave_sum(int64_t lo, int64_t hi) const {
        double s = 0.0;
        if (lo < hi) s = q ? lane_sum<true>(lo, (int)(hi - lo)) : lane_sum<false>(lo, (int)(hi - lo));
        return lane_value(lane_prefix(s), 63);
    }
    // One lane's share: adjacent lanes read adjacent elements, 16 rounds of
    // them in flight (none conditional): any alignment of the row is as good
    // as another, and the body stays small (it runs a few times per launch).
    template <bool Q>
    __device__ __forceinline__ double lane_sum(int64_t lo, int len) const {
        constexpr int U = 16;
        const T *pl = p + lo, *ql = Q ? q + lo : nullptr;
        const int z = zeroed >= lo && zeroed < lo + len ? (int)(zeroed - lo) : -1;
        double s = 0.0;
#pragma unroll 1
        for (int at = threadIdx.x & 63; at < len; at += 64 * U) {
            T pv[U], qv[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int v = min(at + 64 * k, len - 1);
                pv[k] = pl[v];
                if (Q) qv[k] = ql[v];
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int v = at + 64 * k;
                const float f = v < len && v != z ? clean(to_f32(pv[k])) : 0.0f;
                s += Q ? rest(f, to_f32(qv[k])) : (double)f;
            }
        }
        return s;
    }
};

__device__ __forceinline__ int drafts_of(const VerifyParams &p, int64_t b) {
    const int m = p.lens ? p.lens[b] : p.drafts;
    return m < 0 ? 0 : (m > p.drafts ? p.drafts : m);
}

// The number of accepted drafts of sequence b: every wave tests them all, 64
// at a time, so that no wave waits for another.
template <typename T>
__device__ __forceinline__ int accepted_drafts(const VerifyParams &p, int64_t b, int m) {
    for (int i0 = 0; i0 < m; i0 += 64) {
        const int i = i0 + (threadIdx.x & 63);
        bool ok = true;
        if (i < m) {
            const int32_t v = p.tok[b * p.drafts + i];
            ok = v >= 0 && v < p.vocab;
            if (ok) {
                const float q =
                    p.draft ? clean(to_f32(reinterpret_cast<const T *>(p.draft)[b * p.d_bs + i * p.d_rs + v])) : 1.0f;
                ok = (double)p.u[b * (p.drafts + 1) + i] * (double)q <
                     (double)clean(to_f32(reinterpret_cast<const T *>(p.target)[b * p.t_bs + i * p.t_rs + v]));
            }
        }
        const uint64_t rejects = __ballot(!ok);
        if (rejects) return i0 + __builtin_ctzll(rejects);
    }
    return m;
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
    __shared__ double part[kSumThreads / 64];
    const int64_t b = blockIdx.y;
    const int m = drafts_of(p, b), n = accepted_drafts<T>(p, b, m);
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
    __shared__ int wave_hit[kWaves], wave_last[kWaves];
    const int64_t b = blockIdx.x, V = p.vocab;
    const int tid = threadIdx.x, lane = tid & 63, K = p.drafts;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = drafts_of(p, b);
    const int32_t drafted = tid < K ? p.tok[b * K + tid] : -1;
    int n;
    if (p.segments > 1) {
        n = p.n_accepted[b];
    } else {
        n = accepted_drafts<T>(p, b, m);
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
        total = lane_value(upto, 63);
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
    double before = seg > 0 ? lane_value(upto, seg - 1) : 0.0;
    int next = (int)(V - 1);  // a row without mass
    if (seg >= 0) {
        const int64_t lo = seg * segment, hi = min(lo + segment, V);
        // The segment again, kEach adjacent elements per thread at most.
        int found = -1, last_mass = -1;
        for (int64_t from = lo; from < hi; from += kThreads * kEach) {
            const int64_t to = min(from + kThreads * kEach, hi);
            const int each = (int)((to - from + kThreads - 1) / kThreads);
            const int64_t a = from + tid * each;
            // Read kEach elements from `at` on, moved back where they would
            // pass the row's end; this thread's are those in [a, a + each).
            const int64_t at = max(min(a, V - kEach), (int64_t)0);
            double x[kEach], s = 0.0;
            r.read(at, V, x);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                x[i] = at + i >= a && at + i < min(a + each, to) ? x[i] : 0.0;
                s += x[i];
            }
            const double pre = lane_prefix(s);
            if (lane == 63) wave_sums[wave] = pre;
            __syncthreads();
            const double ends = lane_prefix(lane < kWaves ? wave_sums[lane] : 0.0);
            // This thread's elements, from the sum before them.
            double sum = before + (wave > 0 ? lane_value(ends, wave - 1) : 0.0) + (pre - s);
            int last = -1, hit = -1;
#pragma unroll
            for (int i = kEach - 1; i >= 0; --i) last = x[i] > 0.0 && last < 0 ? (int)(at + i) : last;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                sum += x[i];
                if (x[i] > 0.0 && sum > cut && hit < 0) hit = (int)(at + i);
            }
            // The first lane with a hit and the last with mass, then the same
            // over the waves (no atomics: one per lane on one address costs
            // 5 us here).
            const uint64_t hits = __ballot(hit >= 0), some_mass = __ballot(last >= 0);
            if (lane == 0) {
                wave_hit[wave] = -1;
                wave_last[wave] = -1;
            }
            if (hits && lane == __builtin_ctzll(hits)) wave_hit[wave] = hit;
            if (some_mass && lane == 63 - __builtin_clzll(some_mass)) wave_last[wave] = last;
            before += lane_value(ends, kWaves - 1);
            __syncthreads();
            for (int w = kWaves - 1; w >= 0; --w) {
                if (wave_hit[w] >= 0) found = wave_hit[w];
                if (wave_last[w] > last_mass) last_mass = wave_last[w];
            }
            if (found >= 0) break;
            __syncthreads();  // the next turn writes wave_sums and these again
        }
        next = found >= 0 ? found : last_mass;
    }
    if (tid == 0) p.next_token[b] = next;
    if (p.tokens)
        for (int i = tid; i <= K; i += kThreads)
            p.tokens[b * (K + 1) + i] = i < n ? (i == tid ? drafted : p.tok[b * K + i]) : i == n ? next : -1;
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
    // Segments for four workgroups per compute unit, of 2048 elements at least
    // (half a round of a workgroup's loads).
    const int64_t want = std::min<int64_t>({kMaxSegments, 1024 / std::max<int64_t>(p.batch, 1), p.vocab / 2048});
    // Two launches pay where a row alone takes three rounds of its workgroup's
    // loads (us with one launch / two: 1 row of 16384 8.0 / 8.2, of 32000 10.1 /
    // 8.4, of 128256 21.9 / 7.9; 64 rows of 64000 17.4 / 11.4) and the rows leave
    // compute units idle (128 rows of 128256 32.9 / 32.2; 256 rows of 50277 15.7 /
    // 22.6).  The rows at which both are even grow with the row's length: 48 to 64
    // rows of 32000 (48 10.0 / 9.7, 64 10.0 / 10.2, 96 10.2 / 10.8), about 110 of
    // 50277 (64 15.3 / 10.7, 96 16.0 / 15.1, 127 17.0 / 17.5), 127 of 128256 (64
    // 30.7 / 18.8, 96 31.3 / 28.5); 64 for all of them leaves up to a quarter
    // between 65 and 110 long rows.
    const int64_t rounds = p.vocab / (kThreads * 16);
    p.segments = want >= 2 && rounds >= 3 && p.batch <= 64 ? (int)want : 1;
    p.segment = (p.vocab + p.segments - 1) / p.segments;
}

hipError_t launch_verify_drafts(const VerifyParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
