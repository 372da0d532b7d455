// kv4_attn.cu -- decode attention over the 4-bit cache: selected pages, or
// every page of a sequence.
//
// For the G query heads of a KV head, over the tokens of the unit's pages,
//   z = q . k,  out = sum_t 2^(z_t - m) v_t / sum_t 2^(z_t - m)
// in one pass with a running reference m (sm_scale, k_scale and log2(e) are one
// factor on z; v_scale is applied to the result).
//
// Work.  The pages of all units form one list; CTA c of the N launched (one for
// each SM) takes the c-th of N equal pieces of it, whatever the sequences'
// lengths, so there is no tail of long sequences and no more than one wave.
// Every CTA sums the units' page counts itself to find its piece.  The warps
// of a CTA take its pages in turn, each through a private ring of slots filled
// by one bulk copy a page, and run ahead across unit boundaries.  Where a
// unit ends (or the piece does), the warps' partial results are merged in
// shared memory; a unit that lies in one CTA is written out at once, the
// parts of others (two a CTA at most: its first and last unit) go through the
// workspace to a second, small launch.
//
// A 16-token tile.  S^T[16 tok x 8 head] = K[16 x D] Q^T and O^T[D x 8] +=
// V^T[D x 16] P^T on mma.sync m16n8k16 in fp16, fp32 accumulation: a group of
// at most eight heads is too few rows for tcgen05 (M >= 64), and the operands
// are made in registers, where mma.sync takes them.
//   - Codes become halves by cvt.rn.f16x2.e2m1x2 (two a byte; measured at 62
//     lanes a clock and SM, as a logic operation), times the scale: exact.  A
//     shared-memory row is read so that all 32 (D = 64: 16) channels of a lane
//     lie in whole scale groups, so one scale conversion serves a token.
//   - The queries are scaled by a power of two a head so that fp16 holds every
//     bf16 bit that matters (what falls below 2^-39 of the largest is lost).
//   - The contraction over tokens wants pairs of tokens in a register, and a
//     byte holds a pair of channels: the codes of two tokens are interleaved
//     nibble by nibble (two logic operations for eight codes) before the
//     conversion, so V needs no layout of its own and a new token is written
//     as whole bytes.
//   - P is kept as fp16 hi + lo.  With G <= 4 the four spare columns of the
//     tile carry the lo part (queries are repeated there, so those lanes hold
//     the same scores), and one product does both; else there are two.
//   - Tokens are visited in the order r ^ ((r >> 1) & 1) within eight, which
//     lets the K rows of a load fall on different banks and leaves V two ways.
// Launched with programmatic dependent launch.
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace kvmm {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
__host__ __device__ constexpr int ring_depth(int D, int T) { return D * T <= 64 * 16 ? 6 : D * T <= 128 * 16 ? 4 : 2; }

struct Shared {
    uint64_t bar[kWarps][6];
    float m[kWarps][8];
    float l[kWarps][8];
    int scan[kWarps];
};

// dynamic shared memory: [rings][partials: kWarps x G x (D + 4) floats][pre: nu + 1 ints]
__host__ __device__ inline size_t part_offset(int D, int T) { return size_t(kWarps) * ring_depth(D, T) * T * (D + D / 8); }
__host__ __device__ inline size_t pre_offset(int D, int T, int G)
{
    return part_offset(D, T) + size_t(kWarps) * G * (D + 4) * sizeof(float);
}
inline size_t smem_bytes(int D, int T, int G, int nu) { return pre_offset(D, T, G) + size_t(nu + 1) * sizeof(int); }

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// first page of CTA c's piece of `total` pages dealt to n CTAs
__host__ __device__ __forceinline__ int piece_start(int total, int c, int n)
{
    return static_cast<int>(static_cast<long long>(total) * c / n);
}

__device__ __forceinline__ int clamped_seq(const Kv4AttnParams& p, int b, bool tell)
{
    const int cap = p.Pmax * p.T;
    int seq = p.seq_len[b];
    if (seq < 0 || seq > cap) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        seq = seq < 0 ? 0 : cap;
    }
    return seq;
}

template <int D, int T, bool DUP>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_kernel(const Kv4AttnParams p)
{
    using Page = Kv4Page<D, T>;
    constexpr int kDepth = ring_depth(D, T);
    constexpr int kWords = D / 32;   // code words of a lane's K row: its 4 * kWords * 2 channels
    constexpr int kTiles = D / 16;   // m-tiles of O^T
    constexpr int kMine = D / 8;     // output channels of a lane's row group
    constexpr int kVWords = D / 64;  // code words of a lane's V token
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.G;
    const int N = gridDim.x, rank = blockIdx.x;
    uint8_t* ring = smem + static_cast<size_t>(warp) * kDepth * Page::kBytes;
    float* part = reinterpret_cast<float*>(smem + part_offset(D, T));
    int* pre = reinterpret_cast<int*>(smem + pre_offset(D, T, G));

    if (tid < kWarps * kDepth) mbar_init(&sh.bar[tid / kDepth][tid % kDepth], 1);
    fence_barrier_init();
    pdl_wait_then_release();

    // ---- the units' first pages in the launch's page list ----------------------------------------------------
    int total = 0;
    for (int base = 0; base < p.nu; base += kThreads) {
        const int i = base + tid;
        int n = 0;
        if (i < p.nu) {
            const int u = p.u0 + i, b = u / p.Hkv, h = u - b * p.Hkv;
            if (p.sel_cnt != nullptr) {
                n = p.sel_cnt[(static_cast<size_t>(b) * p.L + p.layer) * p.Hkv + h];
                if (n < 0 || n > p.Kmax) {
                    if (rank == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
                    n = n < 0 ? 0 : p.Kmax;
                }
            } else {
                n = (clamped_seq(p, b, rank == 0 && h == 0) + T - 1) / T;
            }
        }
        int inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(kFullMask, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        int before = total, sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int s = sh.scan[w];
            if (w < warp) before += s;
            sum += s;
        }
        if (i < p.nu) pre[i] = before + inc - n;
        total += sum;
        __syncthreads();
    }
    if (tid == 0) pre[p.nu] = total;
    __syncthreads();
    if (rank == 0)
        for (int i = tid; i <= p.nu; i += kThreads) p.pre[i] = pre[i];
    // units without a page: their results are written here, spread over the CTAs
    for (int i = rank * kWarps + warp; i < p.nu; i += N * kWarps) {
        if (pre[i + 1] != pre[i]) continue;
        const int u = p.u0 + i;
        float* o = p.out + static_cast<size_t>(u) * G * D;
        for (int e = lane; e < G * D; e += 32) o[e] = 0.f;
        if (p.lse && lane < G) p.lse[static_cast<size_t>(u) * G + lane] = -INFINITY;
    }
    const int lo = piece_start(total, rank, N), hi = piece_start(total, rank + 1, N);
    if (lo >= hi) return;
    // the last unit that starts at or before a page of the list (empty units share their start with the next)
    auto unit_of = [&](int f) {
        int a = 0, z = p.nu - 1;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (pre[m] <= f) a = m;
            else z = m - 1;
        }
        return a;
    };

    // ---- this warp's pages: lo + warp, lo + warp + kWarps, ... ------------------------------------------------
    int next = lo + warp;        // first page of the batch not looked up yet
    unsigned mask = 0u;          // pages of the batch not issued yet; lane i holds the i-th one's entry
    int e_phys = 0, e_nv = 0, e_u = 0;
    int issued = 0, consumed = 0;
    int s_nv = 0, s_u = 0;       // lane s: valid tokens and unit of the page in slot s
    const uint64_t policy = l2_policy_evict_first();
    auto look_up = [&]() {
        const int f = next + kWarps * lane;
        e_phys = -1;
        if (f < hi) {
            e_u = unit_of(f);
            const int u = p.u0 + e_u, b = u / p.Hkv, h = u - b * p.Hkv;
            const size_t unit = (static_cast<size_t>(b) * p.L + p.layer) * p.Hkv + h;
            const int i = f - pre[e_u];
            const int seq = clamped_seq(p, b, false);
            const int lp = p.sel_idx != nullptr ? p.sel_idx[unit * p.Kmax + i] : i;
            if (lp < 0 || lp >= (seq + T - 1) / T) {
                report(p.err, KVMM_ERR_OUT_OF_RANGE);
            } else {
                const int32_t phys = p.block_table[unit * p.Pmax + lp];
                if (phys < 0 || phys >= p.n_phys) report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
                else e_phys = phys;
                e_nv = min(T, seq - lp * T);
            }
        }
        mask = __ballot_sync(kFullMask, e_phys >= 0);
        next += kWarps * 32;
    };
    auto fill = [&]() {  // issue pages while slots are free
        while (issued - consumed < kDepth) {
            while (mask == 0u) {
                if (next >= hi) return;
                look_up();
            }
            const int src = __ffs(mask) - 1;
            mask &= mask - 1u;
            const int phys = __shfl_sync(kFullMask, e_phys, src);
            const int nv = __shfl_sync(kFullMask, e_nv, src);
            const int u = __shfl_sync(kFullMask, e_u, src);
            const int slot = issued % kDepth;
            if (lane == slot) {
                s_nv = nv;
                s_u = u;
            }
            if (lane == 0) {
                uint64_t* bar = &sh.bar[warp][slot];
                mbar_arrive_expect_tx(bar, Page::kBytes);
                bulk_copy_g2s_hint(ring + slot * Page::kBytes, p.kv4_pool + static_cast<size_t>(phys) * Page::kBytes,
                                   Page::kBytes, bar, policy);
            }
            ++issued;
        }
    };
    fill();

    const int head = DUP ? (gid & 3) : gid;  // the query head of this lane's column
    const int col0 = DUP ? ((2 * tig) & 3) : 2 * tig;  // ... and of its two accumulator columns: col0, col0 + 1
    const int ra = gid ^ ((gid >> 1) & 1);   // the tokens of this lane's K rows: ra and ra + 8
    const int t0 = (2 * tig) ^ (tig & 1), t1 = t0 ^ 1;  // ... and of its V pairs: (t0, t1) and (t0 + 8, t1 + 8)
    bool dead = false;  // a copy never arrived: this warp takes no more pages
    int dead_at = 0;

    for (int u = unit_of(lo); u < p.nu && pre[u] < hi; ++u) {
        const int ubeg = pre[u], uend = pre[u + 1];
        if (uend == ubeg) continue;
        // queries: halves of the lane's channels of its head, scaled by a power of two
        uint32_t qf[2 * kTiles];
        float zf0, zf1;
        {
            const kvmm_bf16* qh = p.q + (static_cast<size_t>(p.u0 + u) * G + head) * D + tig * (D / 4);
            uint4 v[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                v[i] = head < G ? reinterpret_cast<const uint4*>(qh)[i] : make_uint4(0u, 0u, 0u, 0u);
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
            }
            mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
            // 2^e <= mx < 2^(e+1), e kept where 2^(14 - e) and its inverse are normal; scaled queries stay below 2^15
            int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
            e = max(e, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) * p.scale_log2;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) qf[4 * i + k] = pack_half2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
            }
            zf0 = __shfl_sync(kFullMask, down, 4 * (col0));
            zf1 = __shfl_sync(kFullMask, down, 4 * (col0 + 1));
        }

        float o[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        while (issued > consumed && __shfl_sync(kFullMask, s_u, consumed % kDepth) == u) {
            const int slot = consumed % kDepth;
            const int nv = __shfl_sync(kFullMask, s_nv, slot);
            const uint8_t* pg = ring + slot * Page::kBytes;
            if (!dead) {
                const bool ok = mbar_wait_bounded(&sh.bar[warp][slot], (consumed / kDepth) & 1);
                if (__any_sync(kFullMask, !ok)) {  // warp-uniform; the remaining pages are dropped
                    dead = true;
                    dead_at = consumed;
                    if (lane == 0) report(p.err, KVMM_ERR_TIMEOUT);
                }
            }
            if (!dead) {
#pragma unroll
                for (int j = 0; j < T; j += 16) {
                    if (j >= nv) break;
                    const bool full = nv - j >= 16;
                    // ---- scores ----------------------------------------------------------------------------
                    float c[2][4] = {};
                    {
                        const uint8_t* ka = pg + (j + ra) * Page::kRow + tig * (D / 8);
                        const uint8_t* kb = ka + 8 * Page::kRow;
                        uint32_t wa[kWords], wb[kWords], sa[kWords], sb[kWords];
                        if (D == 128) {
                            const uint4 x = ld_shared_v4(ka), y = ld_shared_v4(kb);
                            wa[0] = x.x, wa[1] = x.y, wa[kWords - 2] = x.z, wa[kWords - 1] = x.w;
                            wb[0] = y.x, wb[1] = y.y, wb[kWords - 2] = y.z, wb[kWords - 1] = y.w;
                            // scale groups 2 tig and 2 tig + 1
                            const uint8_t* sc = pg + Page::kKeyScales + (j + ra) * Page::kGroups + 2 * tig;
                            const uint32_t ha = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sc));
                            const uint32_t hb = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sc + 8 * Page::kGroups));
                            sa[0] = sa[1] = prmt(ha, ha, 0x1010);
                            sa[kWords - 2] = sa[kWords - 1] = prmt(ha, ha, 0x3232);
                            sb[0] = sb[1] = prmt(hb, hb, 0x1010);
                            sb[kWords - 2] = sb[kWords - 1] = prmt(hb, hb, 0x3232);
                        } else {
                            const uint2 x = ld_shared_v2(ka), y = ld_shared_v2(kb);
                            wa[0] = x.x, wa[1] = x.y, wb[0] = y.x, wb[1] = y.y;
                            const uint8_t* sc = pg + Page::kKeyScales + (j + ra) * Page::kGroups + tig;
                            const uint32_t h = e4m3x2_to_half2(sc[0] | (static_cast<uint32_t>(sc[8 * Page::kGroups]) << 8));
                            sa[0] = sa[1] = prmt(h, h, 0x1010);
                            sb[0] = sb[1] = prmt(h, h, 0x3232);
                        }
#pragma unroll
                        for (int w = 0; w < kWords; ++w) {
                            mma_f16_16816(c[0], half2_mul(e2m1x2_to_half2<0>(wa[w]), sa[w]),
                                          half2_mul(e2m1x2_to_half2<0>(wb[w]), sb[w]),
                                          half2_mul(e2m1x2_to_half2<1>(wa[w]), sa[w]),
                                          half2_mul(e2m1x2_to_half2<1>(wb[w]), sb[w]), qf[4 * w], qf[4 * w + 1]);
                            mma_f16_16816(c[1], half2_mul(e2m1x2_to_half2<2>(wa[w]), sa[w]),
                                          half2_mul(e2m1x2_to_half2<2>(wb[w]), sb[w]),
                                          half2_mul(e2m1x2_to_half2<3>(wa[w]), sa[w]),
                                          half2_mul(e2m1x2_to_half2<3>(wb[w]), sb[w]), qf[4 * w + 2], qf[4 * w + 3]);
                        }
                    }
                    // x: token ra with heads col0, col0 + 1, then token ra + 8
                    float x[4] = {(c[0][0] + c[1][0]) * zf0, (c[0][1] + c[1][1]) * zf1, (c[0][2] + c[1][2]) * zf0,
                                  (c[0][3] + c[1][3]) * zf1};
                    if (!full) {  // selected, not multiplied: what the page holds there may be anything
                        if (j + ra >= nv) x[0] = x[1] = -INFINITY;
                        if (j + ra + 8 >= nv) x[2] = x[3] = -INFINITY;
                    }
                    // ---- probabilities against a reference per head, raised only when a score exceeds it by
                    // more than kSlack (one vote instead of a reduction a tile).  The reference lies kLift below
                    // the maximum it was taken from, so a probability is at most 2^(kSlack + kLift) = 2^15, and
                    // fp16 hi + lo holds it to 2^-22 of itself or 2^-25 * 2^-kLift of the largest.
                    constexpr float kSlack = 8.f, kLift = 7.f;
                    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
                    if (!__all_sync(kFullMask, mx0 - kLift <= m0 + kSlack && mx1 - kLift <= m1 + kSlack)) {
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) {
                            mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, off));
                            mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, off));
                        }
                        const float n0 = fmaxf(m0, mx0 - kLift), n1 = fmaxf(m1, mx1 - kLift);
                        const float a0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                        const float a1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
                        l0 *= a0;
                        l1 *= a1;
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) {
                            o[i][0] *= a0;
                            o[i][1] *= a1;
                            o[i][2] *= a0;
                            o[i][3] *= a1;
                        }
                        m0 = n0;
                        m1 = n1;
                    }
                    const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
                    const float p0 = fast_exp2(x[0] - r0), p1 = fast_exp2(x[1] - r1);
                    const float p2 = fast_exp2(x[2] - r0), p3 = fast_exp2(x[3] - r1);
                    l0 += p0 + p2;
                    l1 += p1 + p3;
                    const uint32_t h01 = pack_half2(p0, p1), h23 = pack_half2(p2, p3);
                    const uint32_t d01 = pack_half2(p0 - half_lo(h01), p1 - half_hi(h01));
                    const uint32_t d23 = pack_half2(p2 - half_lo(h23), p3 - half_hi(h23));
                    uint32_t b0, b1, e0 = 0u, e1 = 0u;
                    if (DUP) {  // columns 0-3 carry hi, 4-7 lo
                        b0 = movmatrix_trans(tig < 2 ? h01 : d01);
                        b1 = movmatrix_trans(tig < 2 ? h23 : d23);
                    } else {
                        b0 = movmatrix_trans(h01);
                        b1 = movmatrix_trans(h23);
                        e0 = movmatrix_trans(d01);
                        e1 = movmatrix_trans(d23);
                    }
                    // ---- values: channels gid * kMine .. + kMine - 1 of tokens t0, t1, t0 + 8, t1 + 8 -----------
                    const uint8_t* vp = pg + Page::kValues + j * Page::kRow + gid * (D / 16);
                    const uint8_t* vs = pg + Page::kValueScales + j * Page::kGroups + gid * kMine / 16;
                    uint32_t w[4][kVWords];
                    uint32_t sc[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = ((k & 1) ? t1 : t0) + (k >> 1) * 8;
                        if (D == 128) {
                            const uint2 y = ld_shared_v2(vp + t * Page::kRow);
                            w[k][0] = y.x;
                            w[k][kVWords - 1] = y.y;
                        } else {
                            w[k][0] = *reinterpret_cast<const uint32_t*>(vp + t * Page::kRow);
                        }
                        sc[k] = vs[t * Page::kGroups];
                        if (!full && j + t >= nv) sc[k] = 0u;  // a scale of zero: codes are always finite
                    }
                    const uint32_t s01 = e4m3x2_to_half2(sc[0] | (sc[1] << 8));
                    const uint32_t s23 = e4m3x2_to_half2(sc[2] | (sc[3] << 8));
                    // byte i of an even / odd word: channel 2i / 2i + 1 of a token pair
                    uint32_t ev01[kVWords], od01[kVWords], ev23[kVWords], od23[kVWords];
#pragma unroll
                    for (int i = 0; i < kVWords; ++i) {
                        ev01[i] = (w[0][i] & 0x0f0f0f0fu) | ((w[1][i] << 4) & 0xf0f0f0f0u);
                        od01[i] = ((w[0][i] >> 4) & 0x0f0f0f0fu) | (w[1][i] & 0xf0f0f0f0u);
                        ev23[i] = (w[2][i] & 0x0f0f0f0fu) | ((w[3][i] << 4) & 0xf0f0f0f0u);
                        od23[i] = ((w[2][i] >> 4) & 0x0f0f0f0fu) | (w[3][i] & 0xf0f0f0f0u);
                    }
                    // tile i: rows gid are channel i of the lane's, rows gid + 8 channel kTiles + i
                    auto tile = [&](auto ic) {
                        constexpr int i = decltype(ic)::value;
                        constexpr int a = i, b = kTiles + i;  // channels
                        constexpr int ba = (a % 8) / 2, bb = (b % 8) / 2;
                        const uint32_t xa = (a & 1) ? od01[a / 8] : ev01[a / 8], xb = (b & 1) ? od01[b / 8] : ev01[b / 8];
                        const uint32_t ya = (a & 1) ? od23[a / 8] : ev23[a / 8], yb = (b & 1) ? od23[b / 8] : ev23[b / 8];
                        const uint32_t a0 = half2_mul(e2m1x2_to_half2<ba>(xa), s01), a1 = half2_mul(e2m1x2_to_half2<bb>(xb), s01);
                        const uint32_t a2 = half2_mul(e2m1x2_to_half2<ba>(ya), s23), a3 = half2_mul(e2m1x2_to_half2<bb>(yb), s23);
                        mma_f16_16816(o[i], a0, a1, a2, a3, b0, b1);
                        if (!DUP) mma_f16_16816(o[i], a0, a1, a2, a3, e0, e1);
                    };
                    tile(std::integral_constant<int, 0>{});
                    tile(std::integral_constant<int, 1>{});
                    tile(std::integral_constant<int, 2>{});
                    tile(std::integral_constant<int, 3>{});
                    if constexpr (kTiles == 8) {
                        tile(std::integral_constant<int, 4>{});
                        tile(std::integral_constant<int, 5>{});
                        tile(std::integral_constant<int, 6>{});
                        tile(std::integral_constant<int, 7>{});
                    }
                }
            }
            ++consumed;
            __syncwarp();
            fence_proxy_async_shared();  // this slot's reads before the copy that refills it
            if (!dead) fill();
        }

        // ---- the unit ends here (or this CTA's piece of it): merge the warps ---------------------------------------
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(kFullMask, l0, off);
            l1 += __shfl_xor_sync(kFullMask, l1, off);
        }
        if (gid == 0 && (!DUP || tig < 2)) {
            sh.m[warp][col0] = m0;
            sh.m[warp][col0 + 1] = m1;
            sh.l[warp][col0] = l0;
            sh.l[warp][col0 + 1] = l1;
        }
        float* mine = part + static_cast<size_t>(warp) * G * (D + 4);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            if (DUP) {  // hi + lo
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] += __shfl_xor_sync(kFullMask, o[i][k], 2);
            }
            if (!DUP || tig < 2) {
                const int d = gid * kMine + i;
                if (col0 < G) {
                    mine[col0 * (D + 4) + d] = o[i][0];
                    mine[col0 * (D + 4) + d + kTiles] = o[i][2];
                }
                if (col0 + 1 < G) {
                    mine[(col0 + 1) * (D + 4) + d] = o[i][1];
                    mine[(col0 + 1) * (D + 4) + d + kTiles] = o[i][3];
                }
            }
        }
        __syncthreads();
        const bool whole = ubeg >= lo && uend <= hi;
        float* slotp = p.partial + (static_cast<size_t>(rank) * 2 + (ubeg < lo ? 0 : 1)) * kv4_partial_floats(D);
        for (int e = tid; e < G * D; e += kThreads) {
            const int g = e / D, d = e - g * D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][g]);
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sh.m[w][g];
                const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
                L = fmaf(sh.l[w][g], f, L);
                O = fmaf(part[(static_cast<size_t>(w) * G + g) * (D + 4) + d], f, O);
            }
            const size_t row = static_cast<size_t>(p.u0 + u) * G + g;
            if (whole) {
                p.out[row * D + d] = L > 0.f ? O * (p.v_scale / L) : 0.f;
                if (d == 0 && p.lse) p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
            } else {
                slotp[e] = O;
                if (d == 0) {
                    slotp[8 * D + g] = M;
                    slotp[8 * D + 8 + g] = L;
                }
            }
        }
        __syncthreads();  // the partials are free again
    }
    if (dead) {  // copies in flight land before the CTA leaves (bounded)
        for (int k = dead_at; k < issued; ++k)
            mbar_wait_bounded(&sh.bar[warp][k % kDepth], (k / kDepth) & 1, 100000000ull);
    }
}

// ---- units that fell on several CTAs: combine their parts ----------------------------------------------------
__global__ void __launch_bounds__(128) kv4_merge_kernel(const Kv4AttnParams p, int N)
{
    pdl_wait_then_release();
    const int i = blockIdx.x;
    const int total = p.pre[p.nu], beg = p.pre[i], end = p.pre[i + 1];
    if (beg == end) return;
    auto owner = [&](int f) {  // the CTA whose piece holds page f
        int c = static_cast<int>(static_cast<long long>(f) * N / total);
        while (piece_start(total, c + 1, N) <= f) ++c;
        while (piece_start(total, c, N) > f) --c;
        return c;
    };
    const int c0 = owner(beg), c1 = owner(end - 1);
    if (c0 == c1) return;  // written by that CTA
    const int G = p.G, D = p.D;
    const size_t stride = kv4_partial_floats(D);
    for (int e = threadIdx.x; e < G * D; e += blockDim.x) {
        const int g = e / D, d = e - g * D;
        float M = -INFINITY;
        for (int c = c0; c <= c1; ++c) {
            const int s = piece_start(total, c, N);
            if (s == piece_start(total, c + 1, N)) continue;  // an empty piece
            M = fmaxf(M, p.partial[(static_cast<size_t>(c) * 2 + (beg < s ? 0 : 1)) * stride + 8 * D + g]);
        }
        float L = 0.f, O = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const int s = piece_start(total, c, N);
            if (s == piece_start(total, c + 1, N)) continue;
            const float* slot = p.partial + (static_cast<size_t>(c) * 2 + (beg < s ? 0 : 1)) * stride;
            const float m = slot[8 * D + g];
            const float f = m == -INFINITY ? 0.f : exp2f(m - M);
            L = fmaf(slot[8 * D + 8 + g], f, L);
            O = fmaf(slot[e], f, O);
        }
        const size_t row = static_cast<size_t>(p.u0 + i) * G + g;
        p.out[row * D + d] = L > 0.f ? O * (p.v_scale / L) : 0.f;
        if (d == 0 && p.lse) p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

template <int D, int T>
cudaError_t launch(Kv4AttnParams p, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static thread_local int sm_dev = -1, sms = 0;
    if (sm_dev != dev) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        sm_dev = dev;
    }
    const bool dup = p.G <= 4;
    void (*kernel)(Kv4AttnParams) = dup ? kv4_attn_kernel<D, T, true> : kv4_attn_kernel<D, T, false>;
    static thread_local int smem_dev[2] = {-1, -1};
    static thread_local size_t smem_have[2] = {0, 0};
    const int units = p.B * p.Hkv;
    for (p.u0 = 0; p.u0 < units; p.u0 += kKv4MaxUnits) {
        p.nu = units - p.u0 < kKv4MaxUnits ? units - p.u0 : kKv4MaxUnits;
        const size_t smem = smem_bytes(D, T, p.G, p.nu);
        e = allow_smem(kernel, smem, smem_dev[dup], smem_have[dup]);
        if (e != cudaSuccess) return e;
        // one CTA an SM, fewer when not every warp would get a page
        const long long most = static_cast<long long>(p.nu) * (p.sel_idx ? p.Kmax : p.Pmax);
        long long n = (most + kWarps - 1) / kWarps;
        if (n > sms) n = sms;
        if (n > kKv4MaxCtas) n = kKv4MaxCtas;
        e = launch_pdl(kernel, dim3(static_cast<unsigned>(n)), dim3(kThreads), smem, stream, p);
        if (e != cudaSuccess) return e;
        if (n > 1) {
            e = launch_pdl(kv4_merge_kernel, dim3(p.nu), dim3(128), 0, stream, p, static_cast<int>(n));
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
