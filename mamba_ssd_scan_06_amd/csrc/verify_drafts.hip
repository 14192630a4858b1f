// Verification of drafted tokens: per sequence the first draft i with
// u_i q_i(tok_i) >= p_i(tok_i), then a token from the residual
// max(p_n - q_n, 0) (p_m when every draft is accepted) by inverse CDF.
//
// Everything that decides is fp64: u q is exact there (24-bit factors), and
// sums of fp32 values keep 29 spare bits, so that the order in which a row is
// summed moves a border between two tokens by 1e-16 of the row's mass only.
// One workgroup per sequence: each thread sums a contiguous piece of the row,
// the pieces' prefix finds the piece that holds the cut, and its thread walks
// it again.
#include "device_common.hpp"
#include "kernels.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// A probability's mass: NaN and negative values count as none.
__device__ __forceinline__ double mass(double v) { return v > 0.0 ? v : 0.0; }

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_drafts_kernel(VerifyParams p) {
    __shared__ double piece[kThreads];
    __shared__ int first_reject, found, last_mass;
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, K = p.drafts;
    const int64_t V = p.vocab;
    const T *target = reinterpret_cast<const T *>(p.target) + b * p.t_bs;
    const T *draft = p.draft ? reinterpret_cast<const T *>(p.draft) + b * p.d_bs : nullptr;
    const int32_t *tok = K > 0 ? p.tok + b * K : nullptr;
    const float *u = p.u + b * (K + 1);
    int m = K;
    if (p.lens) {
        m = p.lens[b];
        m = m < 0 ? 0 : (m > K ? K : m);
    }
    if (tid == 0) {
        first_reject = m;
        found = 0x7fffffff;
        last_mass = -1;
    }
    __syncthreads();
    for (int i = tid; i < m; i += kThreads) {
        const int32_t v = tok[i];
        bool ok = v >= 0 && v < V;
        if (ok) {
            const double q = draft ? (double)to_f32(draft[i * p.d_rs + v]) : 1.0;
            ok = (double)u[i] * q < (double)to_f32(target[i * p.t_rs + v]);
        }
        if (!ok) atomicMin(&first_reject, i);
    }
    __syncthreads();
    const int n = first_reject;
    const T *pr = target + n * p.t_rs;
    const T *qr = n < m && draft ? draft + n * p.d_rs : nullptr;
    const int64_t zeroed = n < m && !draft ? (int64_t)tok[n] : -1;
    const int64_t per = (V + kThreads - 1) / kThreads, lo = tid * per, hi = lo + per < V ? lo + per : V;
    bool residual = n < m;
    double total = 0.0, before = 0.0;
    auto value = [&](int64_t v) {
        const double pv = (double)to_f32(pr[v]);
        if (!residual) return mass(pv);
        if (qr) return mass(pv - (double)to_f32(qr[v]));
        return v == zeroed ? 0.0 : mass(pv);
    };
    for (int pass = 0; pass < 2; ++pass) {
        double sum = 0.0;
        for (int64_t v = lo; v < hi; ++v) sum += value(v);
        piece[tid] = sum;
        __syncthreads();
        total = 0.0;
        for (int k = 0; k < kThreads; ++k) {
            if (k == tid) before = total;
            total += piece[k];
        }
        __syncthreads();
        if (total > 0.0 || !residual) break;
        residual = false;  // rounding left no mass: p_n itself
    }
    const double cut = (double)u[K] * total;
    double run = before;
    int mine = -1;
    for (int64_t v = lo; v < hi; ++v) {
        const double r = value(v);
        if (r > 0.0) mine = (int)v;
        run += r;
        if (run > cut) {
            atomicMin(&found, (int)v);
            break;
        }
    }
    if (mine >= 0) atomicMax(&last_mass, mine);
    __syncthreads();
    // Rounding (or a uniform outside [0,1)) may leave no such token: the last
    // one with mass, or V-1 for a row without any.
    const int next = found != 0x7fffffff ? found : last_mass >= 0 ? last_mass : (int)(V - 1);
    if (tid == 0) {
        p.n_accepted[b] = n;
        p.next_token[b] = next;
    }
    if (p.tokens)
        for (int i = tid; i <= K; i += kThreads) p.tokens[b * (K + 1) + i] = i < n ? tok[i] : i == n ? next : -1;
}

template <typename T>
hipError_t run(const VerifyParams &p, hipStream_t stream) {
    verify_drafts_kernel<T><<<(unsigned)p.batch, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_drafts(const VerifyParams &p, Elem e, hipStream_t stream) {
    return e == Elem::BF16 ? run<bf16>(p, stream) : run<float>(p, stream);
}

}  // namespace ssd
