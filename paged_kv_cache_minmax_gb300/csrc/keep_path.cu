// keep_path.cu -- after a tree of drafted tokens is verified: the accepted
// nodes' keys and values move to the end of the settled tokens, and the MinMax
// of the pages there are taken from kept rows alone.
//
// A warp takes 32 channels of one (batch, layer, KV head), from the rows' move to
// the pages' bounds: channels do not meet, so no warp waits for another.  The
// pages that rows come from or go to, and those whose bounds are taken, come to
// shared memory in one go (keys by asynchronous copies, values, whose rows are
// channels, by way of registers); rows move there, in order: a row's new place is
// never behind its old one, so every row that is still to move is as it was.
#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {

constexpr int kKeepThreads = 64;  // (two warps: at most 25 KB of shared memory a block)

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

__device__ __forceinline__ void copy16_async(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// shared memory of a warp: the window's key rows (64 bytes each), then each lane's value slots and one word more, so that
// consecutive lanes reach consecutive banks
__host__ __device__ constexpr int keep_key_bytes(int window, int T) { return window * T * 64; }
__host__ __device__ constexpr int keep_warp_bytes(int window, int T)
{
    return keep_key_bytes(window, T) + (window * (T / 2) + 1) * 128;
}

template <int D, int T>
__global__ void __launch_bounds__(kKeepThreads) keep_path_kernel(const KeepParams p, int window)
{
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kShares = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * (kKeepThreads / 32) + warp, part = item % kShares, lh = item / kShares;
    if (lh >= static_cast<unsigned>(p.layers) * static_cast<unsigned>(p.Hkv)) return;
    const int h = lh % p.Hkv, li = lh / p.Hkv, b = blockIdx.y;
    uint8_t* keys = smem + warp * keep_warp_bytes(window, T);
    uint32_t* own = reinterpret_cast<uint32_t*>(keys + keep_key_bytes(window, T)) + lane * (window * (T / 2) + 1);
    uint16_t* slot = reinterpret_cast<uint16_t*>(own);
    pdl_wait_then_release();
    const int cap = p.Pmax * T;
    const int seq = p.seq_len[b], m = p.path_len[b];
    const bool tell = item == 0;  // a sequence's faults are told by one warp
    const int32_t* path = p.path + static_cast<size_t>(b) * p.n_max;
    // nodes of the rows lane and lane + 32
    const int a0 = lane < p.n_max ? path[lane] : 0, a1 = lane + 32 < p.n_max ? path[lane + 32] : 0;
    if (seq < 0 || seq > cap || m < 0 || m > p.n_max) {
        if (tell && lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer0 + li) * p.Hkv + h;
    const int first = seq / T, s0 = seq % T, end = min(seq + m, cap);
    // the window's pages, a lane each
    const int32_t phys = lane < window && first + lane < p.Pmax ? p.block_table[unit * p.Pmax + first + lane] : -1;
    const int up0 = __shfl_up_sync(kFullMask, a0, 1), top = __shfl_sync(kFullMask, a0, 31);
    int up1 = __shfl_up_sync(kFullMask, a1, 1);
    if (lane == 0) up1 = top;
    const bool bad = (lane < m && (a0 >= p.n_max || a0 <= (lane ? up0 : -1))) || (lane + 32 < m && (a1 >= p.n_max || a1 <= up1));
    if (__any_sync(kFullMask, bad)) {
        if (tell && lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    const uint32_t there = __ballot_sync(kFullMask, phys >= 0 && phys < p.n_phys);
    // rows that move, and the pages that they need, come from and go to
    uint64_t moves = 0;
    uint32_t need = 0, values = 0, dest = 0;
    bool beyond = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = lane + 32 * k, come = s0 + (k ? a1 : a0), go = s0 + j;
        bool move = j < m && come != go;
        if (move && first * T + come >= cap) {
            beyond = true;
            move = false;
        }
        const uint32_t pages = move ? 1u << (come / T) | 1u << (go / T) : 0;
        need |= __reduce_or_sync(kFullMask, pages);
        move &= (there & pages) == pages;
        values |= __reduce_or_sync(kFullMask, move ? pages : 0);
        dest |= __reduce_or_sync(kFullMask, move ? 1u << (go / T) : 0);
        moves |= static_cast<uint64_t>(__ballot_sync(kFullMask, move)) << (32 * k);
    }
    const uint32_t bounds = __ballot_sync(kFullMask, p.meta != nullptr && lane < window && (first + lane) * T < end);
    if (part == 0) {
        if (beyond && tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        if (((need | bounds) >> lane & 1) && !(there >> lane & 1))
            report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
    }
    const int d = part * 32 + lane, row8 = lane >> 2, ch = part * 4 + (lane & 3);  // keys: eight rows at once, four lanes a row
    auto page_of = [&](int w) { return static_cast<size_t>(__shfl_sync(kFullMask, phys, w)) * (T * D); };
    for (uint32_t left = (values | bounds) & there; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1;
        const kvmm_bf16* src = p.k_pool + page_of(w) + row8 * D + ch * 8;
#pragma unroll
        for (int i = 0; i < T; i += 8) copy16_async(keys + (w * T + i + row8) * 64 + (lane & 3) * 16, src + i * D);
    }
    for (uint32_t left = values; left != 0;) {  // two pages at once
        const int w0 = __ffs(left) - 1;
        left &= left - 1;
        const int w1 = left != 0 ? __ffs(left) - 1 : w0;
        left &= left - 1;
        const uint4* src0 = reinterpret_cast<const uint4*>(p.v_pool + page_of(w0) + d * T);
        const uint4* src1 = reinterpret_cast<const uint4*>(p.v_pool + page_of(w1) + d * T);
        uint4 v[2][T / 8];
#pragma unroll
        for (int i = 0; i < T / 8; ++i) v[0][i] = src0[i];
#pragma unroll
        for (int i = 0; i < T / 8; ++i) v[1][i] = src1[i];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < T / 8; ++i) {
                uint32_t* o = own + (k ? w1 : w0) * (T / 2) + 4 * i;
                o[0] = v[k][i].x;
                o[1] = v[k][i].y;
                o[2] = v[k][i].z;
                o[3] = v[k][i].w;
            }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // the rows that are left, eight at once: all are read before the first is written
    for (uint64_t left = moves; left != 0;) {
        int row[8], from[8], mine = -1, come = 0;
        uint16_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            row[i] = __ffsll(static_cast<long long>(left)) - 1;  // (none left: -1)
            left &= left - 1;
            from[i] = s0 + __shfl_sync(kFullMask, row[i] < 32 ? a0 : a1, row[i] & 31);
            if (i == row8) {
                mine = row[i];
                come = from[i];
            }
            v[i] = 0;
            if (row[i] >= 0) v[i] = slot[from[i]];
        }
        uint4 k = make_uint4(0, 0, 0, 0);
        if (mine >= 0) k = *reinterpret_cast<const uint4*>(keys + come * 64 + (lane & 3) * 16);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row[i] >= 0) slot[s0 + row[i]] = v[i];
        const int go = s0 + max(mine, 0);
        const int to = __shfl_sync(kFullMask, phys, go / T);
        if (mine >= 0) {
            *reinterpret_cast<uint4*>(keys + go * 64 + (lane & 3) * 16) = k;
            reinterpret_cast<uint4*>(p.k_pool + (static_cast<size_t>(to) * T + go % T) * D)[ch] = k;
        }
        __syncwarp();
    }
    for (uint32_t left = dest; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1;
        uint4* dst = reinterpret_cast<uint4*>(p.v_pool + page_of(w) + d * T);
#pragma unroll
        for (int i = 0; i < T / 8; ++i) {
            const uint32_t* o = own + w * (T / 2) + 4 * i;
            dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    // bounds of the pages up to the new end
    for (uint32_t left = bounds & there; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1, n_valid = min(T, end - (first + w) * T);
        uint32_t lo[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        uint32_t hi[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < T; i += 8) {
            if (i + row8 >= n_valid) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(keys + (w * T + i + row8) * 64 + (lane & 3) * 16);
            const uint32_t k[4] = {to_key2(v.x), to_key2(v.y), to_key2(v.z), to_key2(v.w)};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                lo[x] = __vminu2(lo[x], k[x]);
                hi[x] = __vmaxu2(hi[x], k[x]);
            }
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                lo[x] = __vminu2(lo[x], __shfl_xor_sync(kFullMask, lo[x], off));
                hi[x] = __vmaxu2(hi[x], __shfl_xor_sync(kFullMask, hi[x], off));
            }
        }
        uint4* mm = reinterpret_cast<uint4*>(p.meta + (unit * p.Pmax + first + w) * 2 * D) + ch;
        if (row8 == 0) mm[0] = make_uint4(from_key2(lo[0]), from_key2(lo[1]), from_key2(lo[2]), from_key2(lo[3]));
        if (row8 == 1) mm[D / 8] = make_uint4(from_key2(hi[0]), from_key2(hi[1]), from_key2(hi[2]), from_key2(hi[3]));
    }
}

template <int D, int T>
cudaError_t launch(const KeepParams& p, cudaStream_t stream)
{
    const int window = (p.n_max + T - 2) / T + 1;  // pages that n_max tokens reach
    const size_t smem = static_cast<size_t>(kKeepThreads / 32) * keep_warp_bytes(window, T);
    // (a warp's 32 channels: layers * Hkv * D / 32 is below 2^33, the blocks' number below 2^31)
    const long long warps = static_cast<long long>(p.layers) * p.Hkv * (D / 32);
    const dim3 grid(static_cast<unsigned>((warps + kKeepThreads / 32 - 1) / (kKeepThreads / 32)), p.B);
    return launch_pdl(keep_path_kernel<D, T>, grid, dim3(kKeepThreads), smem, stream, p, window);
}

}  // namespace

cudaError_t launch_keep_path(const KeepParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
