// draft_verify.cu -- which path of each sequence's tree of drafted tokens the
// target's probabilities accept, and the token that follows it.
//
// A child of token x is accepted with probability min(1, w(x) / c(x)); a
// rejected one leaves the residual max(w - c, 0), normalised by its sum W in
// the next factor f = W / Q.  Probabilities are held as whole multiples of
// 2^-53, so the sums over V entries do not depend on how they are split.  No
// residual is stored: an entry's is found again from p, q and the factors of
// the children rejected before it at the same node.
//
// One CTA takes one sequence.  Each warp owns a run of entries, so that the
// drawn token is found from the warps' sums and one warp's second look.
#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {

constexpr int kVerThreads = 1024;
constexpr int kVerWarps = kVerThreads / 32;
constexpr long long kWhole = 1ll << 53;

// floor(x * 2^53) of x clamped to [0, 512] (NaN: 0)
__device__ __forceinline__ long long weight_of(float x)
{
    const uint32_t u = __float_as_uint(x);
    if (!(x > 0.f)) return 0;
    if (x >= 512.f) return 1ll << 62;
    const int e = static_cast<int>(u >> 23);  // x = m * 2^(e - 150), m with its hidden bit
    const unsigned long long m = (u & 0x7fffffu) | 0x800000u;
    if (e >= 97) return static_cast<long long>(m << (e - 97));
    return e > 97 - 24 ? static_cast<long long>(m >> (97 - e)) : 0;
}

struct Row {  // the residual at a node
    const float* p;
    const float* q;    // null: certain candidates
    int rejected;      // children rejected so far
    const float* f;    // their factors, or
    const int* gone;   // with certain candidates, their tokens
};

__device__ __forceinline__ long long residual(const Row& r, float p, float q, int x)
{
    long long w = weight_of(p);
    if (r.q != nullptr) {
        for (int k = 0; k < r.rejected; ++k) {
            w -= weight_of(__fmul_rn(q, r.f[k]));
            w = w < 0 ? 0 : w;
        }
    } else {
        for (int k = 0; k < r.rejected; ++k) w = r.gone[k] == x ? 0 : w;
    }
    return w;
}

__device__ __forceinline__ long long residual_at(const Row& r, int x)
{
    return residual(r, r.p[x], r.q != nullptr ? r.q[x] : 0.f, x);
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

// the sum of a row's residual; every warp's part stays in part[]
__device__ long long row_sum(const Row& r, int V, int run, long long* part)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long first = static_cast<long long>(warp) * run;
    const int end = static_cast<int>(min(first + run, static_cast<long long>(V)));
    long long s = 0;
    for (long long x = first + lane; x < end; x += 32) s += residual_at(r, static_cast<int>(x));
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) part[warp] = s;
    __syncthreads();
    s = part[lane];
    return warp_sum(s);
}

__global__ void __launch_bounds__(kVerThreads) draft_verify_kernel(const VerifyParams p)
{
    __shared__ int token[kTreeMaxNodes], parent[kTreeMaxNodes], path[kTreeMaxNodes], gone[kTreeMaxNodes];
    __shared__ float u[kTreeMaxNodes], factor[kTreeMaxNodes];
    __shared__ long long part[kVerWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x;
    const size_t at = static_cast<size_t>(b) * p.n_max;
    pdl_wait_then_release();
    int n = p.n_nodes != nullptr ? p.n_nodes[b] : p.n_max;
    if (n < 0 || n > p.n_max) {
        if (tid == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        n = n < 0 ? 0 : p.n_max;
    }
    if (tid < n) {
        int t = p.tokens[at + tid], from = p.parent[at + tid];
        if (tid == 0) {
            from = -1;
        } else if (t < 0 || t >= p.V || from < 0 || from >= tid) {
            report(p.err, KVMM_ERR_OUT_OF_RANGE);
            t = 0;
            from = -1;
        }
        token[tid] = t;
        parent[tid] = from;
        u[tid] = p.u_accept[at + tid];
    }
    __syncthreads();
    const int run = ((p.V + kVerWarps - 1) / kVerWarps + 31) & ~31;
    int len = 0, drawn = -1;
    if (n > 0) {
        int cur = 0;
        len = 1;
        if (tid == 0) path[0] = 0;
        Row r{p.target + at * p.target_stride, p.draft != nullptr ? p.draft + at * p.draft_stride : nullptr, 0, factor,
              gone};
        long long W = kWhole;
        double Q = 1.0;
        for (int i = 1; i < n; ++i) {
            if (parent[i] != cur) continue;
            const int x = token[i];
            const long long w = residual_at(r, x);
            long long c = W;
            float f = 0.f, q = 0.f;
            if (r.q != nullptr) {
                q = r.q[x];
                if (W > 0 && Q > 0.0) f = static_cast<float>(static_cast<double>(W) * 0x1p-53 / Q);
                c = weight_of(__fmul_rn(q, f));
            }
            if (static_cast<double>(u[i]) * static_cast<double>(c) < static_cast<double>(w)) {
                cur = i;
                if (tid == 0) path[len] = i;
                ++len;
                r.p = p.target + (at + i) * p.target_stride;
                if (r.q != nullptr) r.q = p.draft + (at + i) * p.draft_stride;
                r.rejected = 0;
                W = kWhole;
                Q = 1.0;
                continue;
            }
            __syncthreads();  // the lists are read above
            if (tid == 0) {
                factor[r.rejected] = f;
                gone[r.rejected] = x;
            }
            __syncthreads();
            ++r.rejected;
            if (r.q != nullptr) {
                W = row_sum(r, p.V, run, part);
                if (p.distinct) Q -= static_cast<double>(q);
            } else {
                W = W > w ? W - w : 0;
            }
        }
        long long sum = row_sum(r, p.V, run, part);
        if (sum == 0) {  // nothing is left: the row itself
            r.rejected = 0;
            sum = row_sum(r, p.V, run, part);
        }
        long long goal = static_cast<long long>(static_cast<double>(p.u_next[b]) * static_cast<double>(sum));
        goal = min(goal, sum - 1);
        // the warp whose run holds the goal, then its entry
        long long before = 0;
        int owner = 0;
        for (; owner < kVerWarps - 1 && before + part[owner] <= goal; ++owner) before += part[owner];
        if (warp == owner) {
            drawn = p.V - 1;
            const long long first = static_cast<long long>(owner) * run;
            for (long long x0 = first; x0 < p.V && x0 < first + run; x0 += 32) {
                const int x = static_cast<int>(x0) + lane;
                long long w = x < p.V && x0 + lane < first + run ? residual_at(r, x) : 0;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const long long y = __shfl_up_sync(kFullMask, w, off);
                    if (lane >= off) w += y;
                }
                const uint32_t over = __ballot_sync(kFullMask, before + w > goal);
                if (over) {
                    drawn = min(p.V - 1, static_cast<int>(x0) + __ffs(over) - 1);
                    break;
                }
                before += __shfl_sync(kFullMask, w, 31);
            }
            if (lane == 0) gone[0] = drawn;
        }
        __syncthreads();
        drawn = gone[0];
    }
    __syncthreads();
    if (tid < p.n_max) {
        p.path[at + tid] = tid < len ? path[tid] : -1;
        p.out_tokens[at + tid] = tid + 1 < len ? token[path[tid + 1]] : tid + 1 == len ? drawn : -1;
    }
    if (tid == 0) p.path_len[b] = len;
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams& p, cudaStream_t stream)
{
    return launch_pdl(draft_verify_kernel, dim3(p.B), dim3(kVerThreads), 0, stream, p);
}

}  // namespace kvmm
