// keep_path.cu -- after a tree of drafted tokens is verified: the accepted
// nodes' keys and values move to the end of the settled tokens, and the MinMax
// of the pages there are taken from kept rows alone.
//
// A CTA takes one (batch, layer, KV head), each warp 32 of its channels: they do not
// meet, so behind the first warp's plan of the moves no warp waits for another.  The
// pages that rows come from or go to, and those whose bounds are taken, come to
// shared memory in one go (keys by asynchronous copies, values, whose rows are
// channels, by way of registers); rows move there, in order: a row's new place is
// never behind its old one, so every row that is still to move is as it was.
//
// 32 sequences, 32 layers, 8 heads, trees of 16: 31 us against 13.9 for the rows' bytes
// at a copy's rate, 17.6 for the sectors they lie in (a value row's are all of its
// page's); bound by waiting for the first warp's plan, by instructions (22 M; 64% of
// the issue slots) and the shared-memory pipe.  One CTA that gathered values two bytes at a time took 67, a
// warp that made its own plan of the moves 33, one that took all channels of a unit
// in turn 38 to 40.  One sequence: 3.8 us, three dependent loads and the launch.
#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {


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

// what the warps of a unit share
struct Plan {
    int moves;                    // rows that move
    uint32_t list[kTreeMaxNodes]; // their old and new slots in the window, in order: old | new << 16
    uint64_t from;                // nodes whose rows move
    uint32_t there, values, dest, bounds;  // pages: in the pools, that moving rows touch, that they go to, whose bounds are taken
    int32_t phys[8];
    int ok;
};

// by the first warp; false: nothing is done to the sequence
template <int T>
__device__ __forceinline__ bool make_plan(const KeepParams& p, int window, int b, size_t unit, bool tell, int seq, int m, Plan& plan)
{
    const int lane = threadIdx.x & 31, cap = p.Pmax * T;
    const int32_t* path = p.path + static_cast<size_t>(b) * p.n_max;
    // nodes of the rows lane and lane + 32
    const int a0 = lane < p.n_max ? path[lane] : 0, a1 = lane + 32 < p.n_max ? path[lane + 32] : 0;
    if (seq < 0 || seq > cap || m < 0 || m > p.n_max) {
        if (tell && lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return false;
    }
    const int first = seq / T, s0 = seq % T, end = min(seq + m, cap);
    // the window's pages, a lane each
    const int32_t phys = lane < window && first + lane < p.Pmax ? p.block_table[unit * p.Pmax + first + lane] : -1;
    const int up0 = __shfl_up_sync(kFullMask, a0, 1), top = __shfl_sync(kFullMask, a0, 31);
    int up1 = __shfl_up_sync(kFullMask, a1, 1);
    if (lane == 0) up1 = top;
    const bool bad = (lane < m && (a0 >= p.n_max || a0 <= (lane ? up0 : -1))) || (lane + 32 < m && (a1 >= p.n_max || a1 <= up1));
    if (__any_sync(kFullMask, bad)) {
        if (tell && lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return false;
    }
    const uint32_t there = __ballot_sync(kFullMask, phys >= 0 && phys < p.n_phys);
    uint64_t from = 0;
    uint32_t need = 0, values = 0, dest = 0;
    int moves = 0;
    bool beyond = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = lane + 32 * k, node = k ? a1 : a0, come = s0 + node, go = s0 + j;
        bool kept = j < m;  // (a row that stays needs its place too)
        if (kept && first * T + come >= cap) {
            beyond = true;
            kept = false;
        }
        const uint32_t pages = kept ? 1u << (come / T) | 1u << (go / T) : 0;
        need |= __reduce_or_sync(kFullMask, pages);
        const bool move = kept && node != j && (there & pages) == pages;
        values |= __reduce_or_sync(kFullMask, move ? pages : 0);
        dest |= __reduce_or_sync(kFullMask, move ? 1u << (go / T) : 0);
        from |= __reduce_or_sync(kFullMask, move && node < 32 ? 1u << node : 0);
        from |= static_cast<uint64_t>(__reduce_or_sync(kFullMask, move && node >= 32 ? 1u << (node - 32) : 0)) << 32;
        const uint32_t those = __ballot_sync(kFullMask, move);
        if (move) plan.list[moves + __popc(those & ((1u << lane) - 1))] = come | go << 16;
        moves += __popc(those);
    }
    const uint32_t bounds = __ballot_sync(kFullMask, p.meta != nullptr && lane < window && (first + lane) * T < end);
    if (beyond && tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
    if (((need | bounds) >> lane & 1) && !(there >> lane & 1))
        report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
    if (lane < window) plan.phys[lane] = phys;
    if (lane == 0) {
        plan.moves = moves;
        plan.from = from;
        plan.there = there;
        plan.values = values;
        plan.dest = dest;
        plan.bounds = bounds & there;
    }
    return true;
}

template <int D, int T>
__global__ void __launch_bounds__(D) keep_path_kernel(const KeepParams p, int window)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Plan plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.Hkv, li = blockIdx.x / p.Hkv, b = blockIdx.y;
    uint8_t* keys = smem + warp * keep_warp_bytes(window, T);
    uint32_t* own = reinterpret_cast<uint32_t*>(keys + keep_key_bytes(window, T)) + lane * (window * (T / 2) + 1);
    uint16_t* slot = reinterpret_cast<uint16_t*>(own);
    pdl_wait_then_release();
    const int seq = p.seq_len[b], m = p.path_len[b];
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer0 + li) * p.Hkv + h;
    if (warp == 0) {
        const bool ok = make_plan<T>(p, window, b, unit, blockIdx.x == 0, seq, m, plan);  // (a sequence's faults are told by one block)
        if (lane == 0) plan.ok = ok;
    }
    __syncthreads();
    if (!plan.ok) return;
    const int first = seq / T, s0 = seq % T, end = min(seq + m, p.Pmax * T);
    const uint32_t values = plan.values, bounds = plan.bounds;
    const uint64_t from = plan.from;
    const int d = warp * 32 + lane, row8 = lane >> 2, ch = warp * 4 + (lane & 3);  // keys: eight rows at once, four lanes a row
    auto page_of = [&](int w) { return static_cast<size_t>(plan.phys[w]) * (T * D); };
    for (uint32_t left = values | bounds; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1;
        const kvmm_bf16* src = p.k_pool + page_of(w) + row8 * D + ch * 8;
#pragma unroll
        for (int i = 0; i < T; i += 8) {
            const int x = w * T + i + row8, node = x - s0;  // rows of the bounds, or that move
            if (x < s0 + m || (node < 64 && (from >> node & 1))) copy16_async(keys + x * 64 + (lane & 3) * 16, src + i * D);
        }
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
    // the rows in order, eight at once: all are read before the first is written
    const int moves = plan.moves;
    for (int j0 = 0; j0 < moves; j0 += 8) {
        uint32_t move[8];
        uint16_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            move[i] = plan.list[min(j0 + i, moves - 1)];  // (the last one again is the same row again)
            v[i] = slot[move[i] & 0xffffu];
        }
        const uint32_t mine = plan.list[min(j0 + row8, moves - 1)], go = mine >> 16;
        const uint4 k = *reinterpret_cast<const uint4*>(keys + (mine & 0xffffu) * 64 + (lane & 3) * 16);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) slot[move[i] >> 16] = v[i];
        if (j0 + row8 < moves) {
            *reinterpret_cast<uint4*>(keys + go * 64 + (lane & 3) * 16) = k;
            reinterpret_cast<uint4*>(p.k_pool + page_of(go / T) + (go % T) * D)[ch] = k;
        }
        __syncwarp();
    }
    for (uint32_t left = plan.dest; left != 0; left &= left - 1) {
        const int w = __ffs(left) - 1;
        uint4* dst = reinterpret_cast<uint4*>(p.v_pool + page_of(w) + d * T);
#pragma unroll
        for (int i = 0; i < T / 8; ++i) {
            const uint32_t* o = own + w * (T / 2) + 4 * i;
            dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    // bounds of the pages up to the new end
    for (uint32_t left = bounds; left != 0; left &= left - 1) {
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
    const int window = (p.n_max + T - 2) / T + 1;  // pages that n_max tokens reach: 5 at most
    const size_t smem = static_cast<size_t>(D / 32) * keep_warp_bytes(window, T);
    static thread_local int dev = -1;
    static thread_local size_t allowed = 0;
    if (smem > 32 * 1024) {  // (49.5 KB at most, beside the plan)
        const cudaError_t e = allow_smem(keep_path_kernel<D, T>, smem, dev, allowed);
        if (e != cudaSuccess) return e;
    }
    // (layers * Hkv is below 2^29: a grid's x, B its y)
    const dim3 grid(static_cast<unsigned>(p.layers) * static_cast<unsigned>(p.Hkv), p.B);
    return launch_pdl(keep_path_kernel<D, T>, grid, dim3(D), smem, stream, p, window);
}

}  // namespace

cudaError_t launch_keep_path(const KeepParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
