// tree_attn.cu -- attention of a tree of drafted tokens over the paged cache.
//
// A warp takes one query row (a node's head): its lanes hold the row's
// channels, and it walks the pages with a running maximum and sum.
#include "common.cuh"
#include "kernels.h"

namespace kvmm {
namespace {

constexpr int kTreeWarps = 8;

template <int D, int T>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_attn_kernel(const TreeAttnParams p)
{
    constexpr int C = D / 32;  // channels of a lane: lane, lane + 32, ..
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z;
    pdl_wait_then_release();
    const int cap = p.Pmax * T;
    const bool tell = blockIdx.x == 0 && warp == 0 && lane == 0;
    int seq = p.seq_len[b], n = p.n_nodes != nullptr ? p.n_nodes[b] : p.n_max;
    if (seq < 0 || seq > cap || n < 0 || n > p.n_max) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        seq = min(max(seq, 0), cap);
        n = min(max(n, 0), p.n_max);
    }
    int held = n;
    if (seq + n > cap) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        held = cap - seq;
    }
    const int row = blockIdx.x * kTreeWarps + warp;
    if (row >= n * p.G) return;
    const int i = row / p.G, g = row % p.G;
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer) * p.Hkv + h;
    const size_t node = static_cast<size_t>(b) * p.n_max + i;
    const size_t at = node * p.Hq + h * p.G + g;
    uint64_t bits = p.tree_mask != nullptr ? p.tree_mask[node] : ~0ull >> (63 - i);
    if (held < 64) bits &= (1ull << held) - 1;
    const int pages = (seq + T - 1) / T;
    int listed = pages, cnt = 0;
    if (p.sel_idx != nullptr) {
        cnt = p.sel_cnt[unit];
        if (cnt < 0 || cnt > p.Kmax) {
            if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
            cnt = min(max(cnt, 0), p.Kmax);
        }
        listed = cnt;
    }
    const int first = seq / T, node_pages = held > 0 ? (seq + held - 1) / T - first + 1 : 0;
    float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        q[c] = __uint_as_float(static_cast<uint32_t>(p.q[at * D + lane + 32 * c]) << 16);
        o[c] = 0.f;
    }
    for (int e = 0; e < listed + node_pages; ++e) {
        const bool settled = e < listed;
        const int page = !settled ? first + e - listed : p.sel_idx != nullptr ? p.sel_idx[unit * p.Kmax + e] : e;
        if (settled && (page < 0 || page >= pages)) {
            if (lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
            continue;
        }
        const int32_t phys = p.block_table[unit * p.Pmax + page];
        if (phys < 0 || phys >= p.n_phys) {
            if (lane == 0) report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
            continue;
        }
        const kvmm_bf16* k = p.k_pool + static_cast<size_t>(phys) * T * D;
        const kvmm_bf16* v = p.v_pool + static_cast<size_t>(phys) * T * D;
        for (int s = 0; s < T; ++s) {
            const int t = page * T + s, j = t - seq;
            const bool live = settled ? j < 0 : j >= 0 && j < held && (bits >> j & 1);
            if (!live) continue;
            float z = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                z = fmaf(q[c], __uint_as_float(static_cast<uint32_t>(k[s * D + lane + 32 * c]) << 16), z);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kFullMask, z, off);
            z *= p.scale_log2;
            const float mn = fmaxf(m, z), f = exp2f(m - mn), w = exp2f(z - mn);
            m = mn;
            l = fmaf(l, f, w);
#pragma unroll
            for (int c = 0; c < C; ++c)
                o[c] = fmaf(o[c], f, w * __uint_as_float(static_cast<uint32_t>(v[(lane + 32 * c) * T + s]) << 16));
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        p.out[at * D + lane + 32 * c] = static_cast<kvmm_bf16>(pack_bf16x2(l > 0.f ? o[c] / l : 0.f, 0.f) & 0xffffu);
    if (p.lse != nullptr && lane == 0) p.lse[at] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t tree_ws_bytes(const kvmm_shape&, int) { return 16; }

cudaError_t launch_tree_attention(const TreeAttnParams& p, cudaStream_t stream)
{
    const dim3 grid((p.n_max * p.G + kTreeWarps - 1) / kTreeWarps, p.Hkv, p.B), block(kTreeWarps * 32);
    if (p.D == 128)
        return p.T == 16 ? launch_pdl(tree_attn_kernel<128, 16>, grid, block, 0, stream, p)
                         : launch_pdl(tree_attn_kernel<128, 32>, grid, block, 0, stream, p);
    return p.T == 16 ? launch_pdl(tree_attn_kernel<64, 16>, grid, block, 0, stream, p)
                     : launch_pdl(tree_attn_kernel<64, 32>, grid, block, 0, stream, p);
}

}  // namespace kvmm
