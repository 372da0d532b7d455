// keep_path.cu -- after a tree of drafted tokens is verified: the accepted
// nodes' keys and values move to the end of the settled tokens, and the MinMax
// of the pages there are taken from kept rows alone.
//
// One CTA takes one (batch, layer, KV head): it reads every row that moves
// into shared memory, then writes them (the rows' old and new places overlap),
// then takes the bounds of the pages, a warp a page.
#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {

constexpr int kKeepThreads = 128;

// bf16 pair -> pair of unsigned 16-bit keys ordered like the values (-0 below +0)
__device__ __forceinline__ uint32_t to_key2(uint32_t w)
{
    const uint32_t neg = (w >> 15) & 0x00010001u;
    return w ^ ((neg * 0xffffu) | 0x80008000u);
}

__device__ __forceinline__ uint32_t from_key2(uint32_t k)
{
    const uint32_t neg = ((~k) >> 15) & 0x00010001u;
    return k ^ ((neg * 0xffffu) | 0x80008000u);
}

template <int D, int T>
__global__ void __launch_bounds__(kKeepThreads) keep_path_kernel(const KeepParams p)
{
    __shared__ uint4 keys[kTreeMaxNodes][D / 8];
    __shared__ uint16_t values[kTreeMaxNodes][D];
    __shared__ int32_t from[kTreeMaxNodes], to[kTreeMaxNodes];  // physical pages, -1: the row does not move
    __shared__ int nodes[kTreeMaxNodes];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.Hkv, li = blockIdx.x / p.Hkv, b = blockIdx.y;
    pdl_wait_then_release();
    const int cap = p.Pmax * T;
    const int seq = p.seq_len[b], m = p.path_len[b];
    const bool tell = blockIdx.x == 0;  // a sequence's faults are told by one CTA
    if (seq < 0 || seq > cap || m < 0 || m > p.n_max) {
        if (tell && tid == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    if (tid < m) nodes[tid] = p.path[static_cast<size_t>(b) * p.n_max + tid];
    __syncthreads();
    const bool bad = tid < m && (nodes[tid] >= p.n_max || nodes[tid] <= (tid ? nodes[tid - 1] : -1));
    if (__syncthreads_or(bad)) {
        if (tell && tid == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer0 + li) * p.Hkv + h;
    const int32_t* table = p.block_table + unit * p.Pmax;
    if (tid < m) {
        const int come = seq + nodes[tid], go = seq + tid;
        int32_t f = -1, t = -1;
        if (come != go) {
            if (come >= cap) {  // (come > go)
                report(p.err, KVMM_ERR_OUT_OF_RANGE);
            } else {
                f = table[come / T];
                t = table[go / T];
                if (f < 0 || t < 0 || f >= p.n_phys || t >= p.n_phys) {
                    if (f < 0 || t < 0) report(p.err, KVMM_ERR_NULL_BLOCK);
                    if (f >= p.n_phys || t >= p.n_phys) report(p.err, KVMM_ERR_OUT_OF_RANGE);
                    f = -1;
                }
            }
        }
        from[tid] = f;
        to[tid] = t;
    }
    __syncthreads();
    for (int i = tid; i < m * (D / 8); i += kKeepThreads) {
        const int j = i / (D / 8), c = i % (D / 8);
        if (from[j] >= 0)
            keys[j][c] = reinterpret_cast<const uint4*>(
                p.k_pool + (static_cast<size_t>(from[j]) * T + (seq + nodes[j]) % T) * D)[c];
    }
    for (int i = tid; i < m * D; i += kKeepThreads) {
        const int j = i / D, d = i % D;
        if (from[j] >= 0) values[j][d] = p.v_pool[(static_cast<size_t>(from[j]) * D + d) * T + (seq + nodes[j]) % T];
    }
    __syncthreads();
    for (int i = tid; i < m * (D / 8); i += kKeepThreads) {
        const int j = i / (D / 8), c = i % (D / 8);
        if (from[j] >= 0)
            reinterpret_cast<uint4*>(p.k_pool + (static_cast<size_t>(to[j]) * T + (seq + j) % T) * D)[c] = keys[j][c];
    }
    for (int i = tid; i < m * D; i += kKeepThreads) {
        const int j = i / D, d = i % D;
        if (from[j] >= 0) p.v_pool[(static_cast<size_t>(to[j]) * D + d) * T + (seq + j) % T] = values[j][d];
    }
    if (p.meta == nullptr) return;
    __syncthreads();

    constexpr int kLanesPerRow = D / 8;
    constexpr int kRowsPerPass = 32 / kLanesPerRow;
    const int end = min(seq + m, cap);
    for (int page = seq / T + warp; page * T < end; page += kKeepThreads / 32) {
        const int32_t phys = table[page];
        if (phys < 0 || phys >= p.n_phys) {
            if (lane == 0) report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
            continue;
        }
        const kvmm_bf16* kpage = p.k_pool + static_cast<size_t>(phys) * T * D;
        const int n_valid = min(T, end - page * T), sub = lane % kLanesPerRow;
        uint32_t lo[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        uint32_t hi[4] = {0u, 0u, 0u, 0u};
        for (int r = lane / kLanesPerRow; r < n_valid; r += kRowsPerPass) {
            const uint4 v = reinterpret_cast<const uint4*>(kpage + static_cast<size_t>(r) * D)[sub];
            const uint32_t w[4] = {to_key2(v.x), to_key2(v.y), to_key2(v.z), to_key2(v.w)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = __vminu2(lo[i], w[i]);
                hi[i] = __vmaxu2(hi[i], w[i]);
            }
        }
#pragma unroll
        for (int off = kLanesPerRow; off < 32; off <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = __vminu2(lo[i], __shfl_xor_sync(kFullMask, lo[i], off));
                hi[i] = __vmaxu2(hi[i], __shfl_xor_sync(kFullMask, hi[i], off));
            }
        }
        if (lane < kLanesPerRow) {
            kvmm_bf16* mm = p.meta + (unit * p.Pmax + page) * 2 * D;
            reinterpret_cast<uint4*>(mm)[lane] =
                make_uint4(from_key2(lo[0]), from_key2(lo[1]), from_key2(lo[2]), from_key2(lo[3]));
            reinterpret_cast<uint4*>(mm + D)[lane] =
                make_uint4(from_key2(hi[0]), from_key2(hi[1]), from_key2(hi[2]), from_key2(hi[3]));
        }
    }
}

}  // namespace

cudaError_t launch_keep_path(const KeepParams& p, cudaStream_t stream)
{
    // (Hkv <= 65535 and the layers of one table: their product is a grid's x, B its y)
    const dim3 grid(static_cast<unsigned>(p.layers) * static_cast<unsigned>(p.Hkv), p.B);
    if (p.D == 128)
        return p.T == 16 ? launch_pdl(keep_path_kernel<128, 16>, grid, dim3(kKeepThreads), 0, stream, p)
                         : launch_pdl(keep_path_kernel<128, 32>, grid, dim3(kKeepThreads), 0, stream, p);
    return p.T == 16 ? launch_pdl(keep_path_kernel<64, 16>, grid, dim3(kKeepThreads), 0, stream, p)
                     : launch_pdl(keep_path_kernel<64, 32>, grid, dim3(kKeepThreads), 0, stream, p);
}

}  // namespace kvmm
