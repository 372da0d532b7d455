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
// A cluster of CTAs takes one sequence.  One lane of each CTA walks the tree (all
// alike; fp64 runs at two lanes a clock); where a sum over the row is needed the
// CTAs share the row, a run of entries for each warp, and exchange their sums
// through distributed shared memory.  The sums of the last pass lead to the drawn
// token: the CTA, the warp, then one look at that warp's run again.
//
// Times (us of a launch in a graph; the floor is the rows drawn from at a copy's rate):
// chains of seven for 64 sequences, 131,072 tokens 23.1 (9.9); trees of 24 certain
// candidates for 16 10.5 (1.2); trees of 16 drawn without replacement for 8, 100,003
// tokens 11 to 27 (0.9) as their random numbers reject: a pass over the row, about 3,
// for every rejected child that has a sibling left; one chain of four, 32,000 tokens
// 6.7 (0.04).  The large case waits for the loads of its pass (a warp's run is four
// rounds of load, wait and sum, at 29% of the memory's rate) and for the one warp
// that looks again; the pass's instructions, 19 an entry, are some 4 of its time.  The
// small ones wait for the chain of loads (the nodes, their probabilities, the row) and
// the cluster's barriers.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerCluster = 16;
constexpr int kStep = 128;  // entries a warp takes at once, four a lane
constexpr int kAhead = 4;   // steps whose loads are in flight
constexpr long long kWhole = 1ll << 53;

// floor(x * 2^53) of x clamped to [0, 512] (NaN: 0).  x = m * 2^(e - 150), m with its hidden bit: m * 2^39 shifted right
// by 136 - e.  (e = 0, a zero or what is far below 2^-53, shifts everything out.)
__device__ __forceinline__ long long weight_of(float x)
{
    const uint32_t u = __float_as_uint(fminf(fmaxf(x, 0.f), 512.f));
    const unsigned long long m = static_cast<unsigned long long>((u << 7) & 0x3fffffffu | 0x40000000u) << 32;
    return static_cast<long long>(m >> min(136u - (u >> 23), 63u));
}

// floor(x * 2^53) of 0 <= x < 2 in three digits: additions that round towards zero leave floor(x * 2^21), floor(r * 2^43)
// of the rest and floor(r * 2^53) of that in the low bits of their results.  (Each rest is exact.)  fp32 additions run at
// twice the rate of the integer pipe's shifts and logic.
constexpr float kDigit1 = 4.f, kDigit2 = 0x1p-20f, kDigit3 = 0x1p-30f;
struct Digits {
    int d1, d2, d3;  // with the bits of kDigit1 .. 3 added
};
__device__ __forceinline__ Digits digits_of(float x)
{
    const float t1 = __fadd_rz(x, kDigit1), r1 = x - (t1 - kDigit1);
    const float t2 = __fadd_rz(r1, kDigit2), r2 = r1 - (t2 - kDigit2);
    return {__float_as_int(t1), __float_as_int(t2), __float_as_int(__fadd_rz(r2, kDigit3))};
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

// entries x .. x + 3 of a row of V, 0 behind its end
__device__ __forceinline__ float4 entries4(const float* row, long long x, int V)
{
    if (x + 4 <= V && (reinterpret_cast<uintptr_t>(row) & 15) == 0) return __ldg(reinterpret_cast<const float4*>(row + x));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x < V) v.x = __ldg(row + x);
    if (x + 1 < V) v.y = __ldg(row + x + 1);
    if (x + 2 < V) v.z = __ldg(row + x + 2);
    if (x + 3 < V) v.w = __ldg(row + x + 3);
    return v;
}

// the residuals of a lane's four entries
__device__ __forceinline__ void residual4(const Row& r, const float4& p, const float4& q, int x, long long (&w)[4])
{
    w[0] = weight_of(p.x);
    w[1] = weight_of(p.y);
    w[2] = weight_of(p.z);
    w[3] = weight_of(p.w);
    if (r.q != nullptr) {
#pragma unroll 1
        for (int k = 0; k < r.rejected; ++k) {
            const float f = r.f[k];
            w[0] = max(w[0] - weight_of(__fmul_rn(q.x, f)), 0ll);
            w[1] = max(w[1] - weight_of(__fmul_rn(q.y, f)), 0ll);
            w[2] = max(w[2] - weight_of(__fmul_rn(q.z, f)), 0ll);
            w[3] = max(w[3] - weight_of(__fmul_rn(q.w, f)), 0ll);
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < r.rejected; ++k) {
            const int at = r.gone[k] - x;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = at == e ? 0 : w[e];
        }
    }
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

struct Shared {
    int token[kTreeMaxNodes], path[kTreeMaxNodes], gone[kTreeMaxNodes];
    float u[kTreeMaxNodes], factor[kTreeMaxNodes];
    float p[kTreeMaxNodes], q[kTreeMaxNodes];          // a node's token in its parent's rows
    unsigned long long children[kTreeMaxNodes];        // bits
    int first[kTreeMaxNodes];                          // whether a node is accepted where it is its parent's first to be tried
    long long part[kVerWarps];                         // the warps' sums of a pass
    long long totals[2][kVerCluster];                  // the CTAs', by the pass's parity
    long long before;                                  // the drawn token's: what lies before its warp's run
    long long goal;
    int owner;                                         // its warp, -1: in another CTA
    float u_next;
    int cur, rejected, len, ask;                       // ask: a sum is wanted for the walk
};

__device__ __forceinline__ void st_cluster_s64(long long* local, uint32_t rank, long long v)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}

// The sum of a row's residual over all CTAs of the cluster; the warps' and the CTAs' parts stay in part and totals.
// A CTA writes totals of the pass after next only behind the next pass's barrier, when all have read these.
__device__ __forceinline__ long long row_sum(const Row& r, int V, int run, int ctas, int parity, Shared& sh)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_ctarank();
    const long long first = static_cast<long long>(rank * kVerWarps + warp) * run;
    const long long end = min(first + run, static_cast<long long>(V));
    long long s = 0;
    // One pass for what is met most, a row as it is and a row less the draft's once: P - Q where p > q and nothing where
    // not, which is P less the weight of min(p, q), as floor() ascends.  19 instructions an entry, most of them fp32,
    // against 46 with every residual in 64 bits: the pass was bound by the integer pipe.
    const bool plain = r.rejected == 0 || r.q == nullptr || r.rejected == 1;
    uint32_t odd = 0;  // of any p or q f an exponent of 2 or more, or a sign: no probability, the general pass is right for it
    if (plain) {
        const float f = r.q != nullptr ? r.f[0] : 0.f;
        // steps of both rows, or twice as many of one, in flight
        auto steps = [&](auto both) {
            constexpr bool kBoth = decltype(both)::value;
            constexpr int kN = kBoth ? kAhead : 2 * kAhead;
#pragma unroll 1
            for (long long x0 = first + 4 * lane; x0 < end; x0 += kN * kStep) {
                float4 p[kN], q[kBoth ? kN : 1];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const long long x = x0 + i * kStep;
                    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (kBoth) q[i] = p[i];
                    if (x < end) {
                        p[i] = entries4(r.p, x, V);
                        if (kBoth) q[i] = entries4(r.q, x, V);
                    }
                }
                int d1 = 0, d2 = 0, d3 = 0;  // 16 entries' digits of 22 bits, or 32 entries', less those of a zero
                const Digits zero = digits_of(0.f);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float pp[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
                    const float4 y = kBoth ? q[kBoth ? i : 0] : p[i];
                    const float qq[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float c = kBoth ? __fmul_rn(qq[k], f) : 0.f;
                        odd |= __float_as_uint(pp[k]) | __float_as_uint(c);
                        const Digits a = digits_of(pp[k]), b = kBoth ? digits_of(fminf(c, pp[k])) : zero;
                        d1 += a.d1 - b.d1;
                        d2 += a.d2 - b.d2;
                        d3 += a.d3 - b.d3;
                    }
                }
                s += (static_cast<long long>(d1) << 32) + (static_cast<long long>(d2) << 10) + d3;
            }
        };
        if (r.q != nullptr)
            steps(std::true_type{});
        else
            steps(std::false_type{});
        if (r.q == nullptr)  // less the rejected candidates, each once
            for (int k = lane; k < r.rejected; k += 32) {
                const int x = r.gone[k];
                bool again = x < first || x >= end;
                for (int e = 0; e < k; ++e) again |= r.gone[e] == x;
                if (!again) s -= weight_of(r.p[x]);
            }
    }
    if (!plain || __any_sync(kFullMask, (odd >> 30) != 0)) {
        s = 0;
#pragma unroll 1
        for (long long x = first + 4 * lane; x < end; x += kStep) {
            const float4 p = entries4(r.p, x, V);
            const float4 q = r.q != nullptr ? entries4(r.q, x, V) : make_float4(0.f, 0.f, 0.f, 0.f);
            long long w[4];
            residual4(r, p, q, static_cast<int>(x), w);
            s += (w[0] + w[1]) + (w[2] + w[3]);
        }
    }
    s = warp_sum(s);
    if (lane == 0) sh.part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        s = warp_sum(lane < kVerWarps ? sh.part[lane] : 0);
        if (lane < ctas) st_cluster_s64(&sh.totals[parity][rank], lane, s);
    }
    cluster_sync();
    s = 0;
    for (int k = 0; k < ctas; ++k) s += sh.totals[parity][k];
    return s;
}

__global__ void __launch_bounds__(kVerThreads, 4) draft_verify_kernel(const VerifyParams p, int ctas, int run)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = cluster_ctarank();
    const int b = blockIdx.x / ctas;
    const size_t at = static_cast<size_t>(b) * p.n_max;
    if (tid < kTreeMaxNodes) sh.children[tid] = 0;
    cluster_arrive();
    pdl_wait_then_release();
    int n = p.n_nodes != nullptr ? p.n_nodes[b] : p.n_max;
    if (n < 0 || n > p.n_max) {
        if (tid == 0 && rank == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        n = n < 0 ? 0 : p.n_max;
    }
    if (n == 0) {  // (the whole cluster leaves)
        if (rank == 0 && tid < p.n_max) p.path[at + tid] = p.out_tokens[at + tid] = -1;
        if (rank == 0 && tid == 0) p.path_len[b] = 0;
        cluster_wait();
        return;
    }
    __syncthreads();
    if (tid < n) {
        const int t = p.tokens[at + tid], from = p.parent[at + tid];
        sh.token[tid] = t;
        sh.u[tid] = p.u_accept[at + tid];
        if (tid > 0) {
            if (t >= 0 && t < p.V && from >= 0 && from < tid) {
                const float pt = p.target[(at + from) * p.target_stride + t];
                const float qt = p.draft != nullptr ? p.draft[(at + from) * p.draft_stride + t] : 0.f;
                const long long c = p.draft != nullptr ? weight_of(qt) : kWhole;
                sh.p[tid] = pt;
                sh.q[tid] = qt;
                sh.first[tid] = static_cast<double>(sh.u[tid]) * static_cast<double>(c) < static_cast<double>(weight_of(pt));
                atomicOr(&sh.children[from], 1ull << tid);
            } else if (rank == 0) {
                report(p.err, KVMM_ERR_OUT_OF_RANGE);
            }
        }
    }
    if (tid == 0) {
        sh.cur = sh.rejected = 0;
        sh.u_next = p.u_next[b];
        sh.path[0] = 0;
        sh.len = 1;
    }
    __syncthreads();
    cluster_wait();  // every CTA of the cluster has begun: its shared memory may be written

    Row r{nullptr, nullptr, 0, sh.factor, sh.gone};
    unsigned long long left = sh.children[0];  // children to be tried (thread 0's)
    long long W = kWhole;
    double Q = 1.0;
    int parity = 0;
    for (;;) {
        if (tid == 0) {
            sh.ask = 0;
            while (left != 0) {
                const int i = __ffsll(static_cast<long long>(left)) - 1, x = sh.token[i];
                left &= left - 1;
                long long w = 0;
                float f = 1.f;  // (of a first child: W / 2^53 and Q are 1)
                bool accepted;
                if (sh.rejected == 0) {
                    accepted = sh.first[i] != 0;
                    w = weight_of(sh.p[i]);
                } else {
                    r.q = p.draft;
                    r.rejected = sh.rejected;
                    w = residual(r, sh.p[i], sh.q[i], x);
                    long long c = W;
                    if (p.draft != nullptr) {
                        f = W > 0 && Q > 0.0 ? static_cast<float>(static_cast<double>(W) * 0x1p-53 / Q) : 0.f;
                        c = weight_of(__fmul_rn(sh.q[i], f));
                    }
                    accepted = static_cast<double>(sh.u[i]) * static_cast<double>(c) < static_cast<double>(w);
                }
                if (accepted) {
                    sh.cur = i;
                    sh.path[sh.len++] = i;
                    sh.rejected = 0;
                    left = sh.children[i];
                    W = kWhole;
                    Q = 1.0;
                    continue;
                }
                sh.factor[sh.rejected] = f;
                sh.gone[sh.rejected] = x;
                ++sh.rejected;
                if (p.draft == nullptr) {
                    W = W > w ? W - w : 0;
                    continue;
                }
                if (p.distinct) Q -= static_cast<double>(sh.q[i]);
                sh.ask = left != 0;
                break;
            }
        }
        __syncthreads();
        const bool more = sh.ask != 0;
        r.p = p.target + (at + sh.cur) * p.target_stride;
        r.rejected = sh.rejected;
        r.q = p.draft != nullptr && r.rejected > 0 ? p.draft + (at + sh.cur) * p.draft_stride : nullptr;
        W = row_sum(r, p.V, run, ctas, parity, sh);  // (its barriers stand between the walk's reads and writes)
        parity ^= 1;
        if (!more) break;
    }
    if (W == 0 && r.rejected > 0) {  // nothing is left: the row itself
        r.rejected = 0;
        r.q = nullptr;
        W = row_sum(r, p.V, run, ctas, parity, sh);
        parity ^= 1;
    }
    if (tid == 0) {  // the CTA whose entries hold the goal, and its warp
        const long long goal = min(static_cast<long long>(static_cast<double>(sh.u_next) * static_cast<double>(W)), W - 1);
        const long long* totals = sh.totals[parity ^ 1];
        long long before = 0;
        int cta = 0, owner = 0;
        for (; cta < ctas - 1 && before + totals[cta] <= goal; ++cta) before += totals[cta];
        for (; cta == rank && owner < kVerWarps - 1 && before + sh.part[owner] <= goal; ++owner) before += sh.part[owner];
        sh.goal = goal;
        sh.before = before;
        sh.owner = cta == rank ? owner : -1;
    }
    __syncthreads();
    if (warp != sh.owner) return;
    const long long goal = sh.goal;
    long long before = sh.before;
    const long long first = static_cast<long long>(rank * kVerWarps + warp) * run;
    const long long end = min(first + run, static_cast<long long>(p.V));
    int drawn = -1;
#pragma unroll 1
    for (long long x0 = first + 4 * lane; x0 - 4 * lane < end && drawn < 0; x0 += kAhead * kStep) {
        float4 pp[kAhead], qq[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const long long x = x0 + i * kStep;
            pp[i] = qq[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < end) {
                pp[i] = entries4(r.p, x, p.V);
                if (r.q != nullptr) qq[i] = entries4(r.q, x, p.V);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int x = static_cast<int>(x0) + i * kStep;
            long long w[4];
            residual4(r, pp[i], qq[i], x, w);
            const long long mine = (w[0] + w[1]) + (w[2] + w[3]);
            long long upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(kFullMask, upto, off);
                if (lane >= off) upto += y;
            }
            const uint32_t over = __ballot_sync(kFullMask, before + upto > goal);
            if (over != 0 && drawn < 0) {
                long long c = before + upto - mine;
                int k = 0;
                for (; k < 3; ++k) {
                    c += w[k];
                    if (c > goal) break;
                }
                drawn = __shfl_sync(kFullMask, min(x + k, p.V - 1), __ffs(over) - 1);
            }
            before += __shfl_sync(kFullMask, upto, 31);
        }
    }
    if (drawn < 0) drawn = p.V - 1;
    const int len = sh.len;
    for (int i = lane; i < p.n_max; i += 32) {
        p.path[at + i] = i < len ? sh.path[i] : -1;
        p.out_tokens[at + i] = i + 1 < len ? sh.token[sh.path[i + 1]] : i + 1 == len ? drawn : -1;
    }
    if (lane == 0) p.path_len[b] = len;
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams& p, cudaStream_t stream)
{
    // As many CTAs a sequence as all run at once (64 registers a thread: four an SM), each with a step of entries for every
    // warp at least.
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static thread_local int known = -1, sms = 0;
    if (known != dev) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(draft_verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        known = dev;
    }
    int ctas = 1;
    while (ctas < kVerCluster && 2ll * ctas * p.B <= 4ll * sms && static_cast<long long>(ctas) * kVerWarps * kStep < p.V) ctas *= 2;
    const long long warps = static_cast<long long>(ctas) * kVerWarps;
    const int run = static_cast<int>((p.V + warps * kStep - 1) / (warps * kStep)) * kStep;
    return launch_pdl_cluster(draft_verify_kernel, dim3(static_cast<unsigned>(p.B) * ctas), dim3(kVerThreads), 0, stream,
                              static_cast<unsigned>(ctas), p, ctas, run);
}

}  // namespace kvmm
