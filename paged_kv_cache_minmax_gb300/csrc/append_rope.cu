// append_rope.cu -- kv_append_rope and kv4_append_rope: new queries, keys and
// values as a projection leaves them; queries and keys rotated by position,
// keys and values written to their pages (bf16, or held in 4 bits) and the
// pages' key MinMax refreshed.
//
// Rotation of a pair of channels: (a, b) -> (a c - b s, b c + a s) in fp32,
// each product and the sum rounded by itself.  A fused multiply-add would
// round once less, but which product it fuses is the compiler's choice; the
// 4-bit codes then depend on it where a value lies next to a border.
//
// One warp takes one page of one (batch, KV head), as in minmax_update.cu: the
// page is the unit of its MinMax and of its table entry.  D/16 lanes share a
// token's row; a lane holds two pieces of eight channels, i and i + dim/2 (in
// the part that does not turn, the piece half of that part further on), so
// both members of every pair are in one lane whichever way channels are
// paired, and the 16 channels of a 4-bit scale are in two neighbouring lanes.
// Rows of the page that were there before are read back (for the MinMax
// alone); where more than two of a block of 16 value rows are new, the block's
// other rows are read and it is stored whole.  Further warps rotate the query
// rows, 16 (D = 64: 32) each with their loads in flight together: the heads of
// one token where its heads are whole blocks, so that its range, position and
// angles are looked up once, else rows of the whole list (32K prompt, 32 heads:
// 133 us by blocks, 137 by rows; two 8K prompts, pages of 32: 71 and 77).
//
// Bound and measured (one GB300): prompts by the bytes they move.  Single tokens
// by a chain of loads: range, table entry, then the begun page's rows in passes
// of which each waits for its loads (D = 128: four, 4-bit pages of 32 eight),
// and after the MinMax the bf16 value row.  A 32K prompt, 32 query and 8 KV
// heads of 128 channels (830 MB): 134 us, 0.91 of a copy's rate; the first
// version, with a store between every two rows' loads and angles for every head,
// took 240.  One token a sequence, batch 32: 5.1 us on the device.  Two chunks of
// 8K tokens into 4 bits 64.5 us (364 MB, 0.83) and, by kv4_gather, back 81 (453
// MB, 0.83); the first version, with a division a channel besides, took 151.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace kvmm {
namespace {

constexpr int kAppWarps = 8;

// bf16 pair -> pair of unsigned 16-bit keys ordered like the values
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

// tokens of [tb, te) this call appends, 0 for a range that is refused
__device__ __forceinline__ int token_count(const AppendParams& p, int tb, int te)
{
    const int cap = p.Pmax * p.T;
    if (tb < 0 || te < tb || tb > cap) return 0;
    return min(min(te, cap) - tb, p.n_new);
}

// the tokens of batch b this call appends: [tb, te), clamped as kv_minmax_update clamps
__device__ __forceinline__ bool token_range(const AppendParams& p, int b, int& tb, int& te, bool tell)
{
    tb = p.tok_begin[b];
    te = p.tok_end[b];
    const int cap = p.Pmax * p.T;
    if (tb < 0 || te < tb || tb > cap) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        return false;
    }
    if (te > cap || te - tb > p.n_new) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        te = min(te, cap);
        if (te - tb > p.n_new) te = tb + p.n_new;
    }
    return te > tb;
}

// the position of row j of batch b (token t), -1 when it lies outside the table
__device__ __forceinline__ int position(const AppendParams& p, int b, int j, int t)
{
    if (p.rope.table == nullptr) return 0;
    const int pos = p.rope.positions ? p.rope.positions[static_cast<size_t>(b) * p.n_new + j] : t;
    return pos >= 0 && pos < p.rope.rows ? pos : -1;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s)
{
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// a lane's pieces: `sub` of the D/16 lanes of a row
struct Pieces {
    int a, b;
    bool turns;
};
template <int D>
__device__ __forceinline__ Pieces pieces(const AppendParams& p, int sub)
{
    const int r = p.rope.table ? p.rope.dim / 16 : 0;  // pieces in half of the part that turns
    if (sub < r) return {sub, sub + r, true};
    const int rest = D / 16 - r;
    return {2 * r + (sub - r), 2 * r + rest + (sub - r), false};
}

// x with its magnitude limited to fp32's largest: an infinity becomes that value of its sign; NaN stays
__device__ __forceinline__ float limited(float x)
{
    float y;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(FLT_MAX));
    return y;
}

// the largest of m, |x| and |y|, NaN if one of them is (fmaxf would drop it, and the channel become a number)
__device__ __forceinline__ float largest(float m, float x, float y)
{
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(x), "f"(y));
    return m;
}

// x / d for finite x, from r = 1/d (rounded): the product and one correction by its residual (Markstein 1990), x/d to
// within 2^-45 before the one rounding.  Where it is taken, what matters is that a quotient that is a border of the
// next, coarser rounding comes out as that border and every other on its side of it: x has 24 significant bits and the
// product of d and a border at most seven, so x/d is off a border by at least 1.01 half-steps of fp32 there, or not at
// all.  The residual is taken as q d - x, so that a zero x, whose residual is +0 either way, keeps its sign.
__device__ __forceinline__ float quotient(float x, float d, float r)
{
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(-__fmaf_rn(q, d, -x), r, q);
}

// Hold a lane's two pieces in 4 bits: codes (eight nibbles a piece) and the
// scales' bytes; `a`, `b` become x / factor.  Every lane of the warp calls.
// A NaN makes the scale NaN (0x7f) and the group's quotients NaN, whose code is 7.
// LIMIT: an infinite x / factor counts as fp32's largest value.  Else it gives a
// wrong scale and codes (the residual of its quotient is NaN), and `most`, the
// running largest magnitude, tells of it.
template <bool LIMIT>
__device__ __forceinline__ void hold4(float (&a)[8], float (&b)[8], float inv, uint32_t& code_a, uint32_t& code_b,
                                      uint32_t& scale_a, uint32_t& scale_b, float& most)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = __fmul_rn(a[i], inv);
        b[i] = __fmul_rn(b[i], inv);
        if (LIMIT) {
            a[i] = limited(a[i]);
            b[i] = limited(b[i]);
        }
    }
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        ma = largest(ma, a[i], a[i + 1]);
        mb = largest(mb, b[i], b[i + 1]);
    }
    if (!LIMIT) most = fmaxf(fmaxf(most, ma), mb);  // (a group with a NaN needs no limits)
    ma = largest(ma, __shfl_xor_sync(kFullMask, ma, 1), 0.f);  // the other eight channels of the scale
    mb = largest(mb, __shfl_xor_sync(kFullMask, mb, 1), 0.f);
    constexpr float kSixth = 1.f / 6.f;
    scale_a = float_to_e4m3(quotient(ma, 6.f, kSixth));
    scale_b = float_to_e4m3(quotient(mb, 6.f, kSixth));
    const uint32_t s2 = e4m3x2_to_half2(scale_a | (scale_b << 8));
    const float sa = half_lo(s2), sb = half_hi(s2);
    const float ra = __frcp_rn(sa), rb = __frcp_rn(sb);
    code_a = code_b = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        code_a |= float2_to_e2m1x2(quotient(a[2 * i], sa, ra), quotient(a[2 * i + 1], sa, ra)) << (8 * i);
        code_b |= float2_to_e2m1x2(quotient(b[2 * i], sb, rb), quotient(b[2 * i + 1], sb, rb)) << (8 * i);
    }
    if (scale_a == 0u) code_a = 0u;
    if (scale_b == 0u) code_b = 0u;
}

// eight codes and their scale -> four bf16 pairs (exact)
__device__ __forceinline__ uint4 held8(uint32_t code, uint32_t scale)
{
    const uint32_t s = e4m3x2_to_half2(scale | (scale << 8));
    const uint32_t h[4] = {half2_mul(e2m1x2_to_half2<0>(code), s), half2_mul(e2m1x2_to_half2<1>(code), s),
                           half2_mul(e2m1x2_to_half2<2>(code), s), half2_mul(e2m1x2_to_half2<3>(code), s)};
    return make_uint4(pack_bf16x2(half_lo(h[0]), half_hi(h[0])), pack_bf16x2(half_lo(h[1]), half_hi(h[1])),
                      pack_bf16x2(half_lo(h[2]), half_hi(h[2])), pack_bf16x2(half_lo(h[3]), half_hi(h[3])));
}

// running order keys of a lane's piece
struct Bounds {
    uint32_t lo[4], hi[4];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = 0xffffffffu;
            hi[i] = 0u;
        }
    }
    __device__ __forceinline__ void add(const uint4& v)
    {
        const uint32_t w[4] = {to_key2(v.x), to_key2(v.y), to_key2(v.z), to_key2(v.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __vminu2(lo[i], w[i]);
            hi[i] = __vmaxu2(hi[i], w[i]);
        }
    }
    __device__ __forceinline__ void across(int off)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __vminu2(lo[i], __shfl_xor_sync(kFullMask, lo[i], off));
            hi[i] = __vmaxu2(hi[i], __shfl_xor_sync(kFullMask, hi[i], off));
        }
    }
    __device__ __forceinline__ void store(kvmm_bf16* m, int D, int piece) const
    {
        reinterpret_cast<uint4*>(m)[piece] = make_uint4(from_key2(lo[0]), from_key2(lo[1]), from_key2(lo[2]), from_key2(lo[3]));
        reinterpret_cast<uint4*>(m + D)[piece] = make_uint4(from_key2(hi[0]), from_key2(hi[1]), from_key2(hi[2]), from_key2(hi[3]));
    }
};

// the angles of a lane's two pieces at one position
struct Angles {
    float4 c0, c1, s0, s1;
};
__device__ __forceinline__ Angles angles(const AppendParams& p, int pos, const Pieces& pc)
{
    const float* cs = p.rope.table + static_cast<size_t>(pos) * p.rope.dim;
    const float* sn = cs + p.rope.dim / 2;
    // pairs inside a piece: angles 4c .. 4c + 3 of either; channel i with i + dim/2: angles 8a .. 8a + 7
    const int i0 = p.rope.interleaved ? pc.a : 2 * pc.a, i1 = p.rope.interleaved ? pc.b : 2 * pc.a + 1;
    return {reinterpret_cast<const float4*>(cs)[i0], reinterpret_cast<const float4*>(cs)[i1],
            reinterpret_cast<const float4*>(sn)[i0], reinterpret_cast<const float4*>(sn)[i1]};
}
__device__ __forceinline__ void rotate(const AppendParams& p, const Angles& g, float (&a)[8], float (&b)[8])
{
    if (p.rope.interleaved) {
        turn(a[0], a[1], g.c0.x, g.s0.x);
        turn(a[2], a[3], g.c0.y, g.s0.y);
        turn(a[4], a[5], g.c0.z, g.s0.z);
        turn(a[6], a[7], g.c0.w, g.s0.w);
        turn(b[0], b[1], g.c1.x, g.s1.x);
        turn(b[2], b[3], g.c1.y, g.s1.y);
        turn(b[4], b[5], g.c1.z, g.s1.z);
        turn(b[6], b[7], g.c1.w, g.s1.w);
    } else {
        turn(a[0], b[0], g.c0.x, g.s0.x);
        turn(a[1], b[1], g.c0.y, g.s0.y);
        turn(a[2], b[2], g.c0.z, g.s0.z);
        turn(a[3], b[3], g.c0.w, g.s0.w);
        turn(a[4], b[4], g.c1.x, g.s1.x);
        turn(a[5], b[5], g.c1.y, g.s1.y);
        turn(a[6], b[6], g.c1.z, g.s1.z);
        turn(a[7], b[7], g.c1.w, g.s1.w);
    }
}

// ... of bf16 rows
__device__ __forceinline__ void turn_row(const AppendParams& p, const Angles& g, uint4& va, uint4& vb)
{
    float a[8], c[8];
    unpack8(va, a);
    unpack8(vb, c);
    rotate(p, g, a, c);
    va = pack8(a);
    vb = pack8(c);
}

constexpr int kQueryPasses = 4;  // rows of one token a lane turns: its loads in flight together

// Loads come before the stores that follow them in each batch: the compiler may not move a load over a store that
// could alias it, so the order written is the number of bytes in flight.
// Rows in flight: one pass a warp with 24 warps an SM (80 registers a thread; the 4-bit kernels spill 32 or 36 bytes,
// the bf16 ones 8 or 36), or two with 16 (no spills).  The first is as fast or faster where the work between load and
// store is long or a page has few passes (32K prompt, pages of 16: 133 us against 143; 336 tokens of 45 sequences into
// 4-bit pages of 32 and back: 39 against 46); bf16 pages of 32 have twice the passes in a chain and little else (short
// prompts: 8.4 us with two at once, 9.9 with one).
template <int T, bool KV4>
constexpr int kAppBatch = T == 16 || KV4 ? 1 : 2;

template <int D, int T, bool KV4>
__global__ void __launch_bounds__(kAppWarps * 32, kAppBatch<T, KV4> == 1 ? 3 : 2)
    append_rope_kernel(const AppendParams p, int page_slots, unsigned kv_ctas, int head_blocks)
{
    using Page = Kv4Page<D, T>;
    constexpr int kLanes = D / 16;      // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows a warp moves at once
    constexpr int kBatch = kAppBatch<T, KV4>;  // passes loaded together
    static_assert(T % (kRows * kBatch) == 0, "whole batches");
    pdl_wait_then_release();  // the pools, table and metadata may be in use by the previous kernel
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int sub = lane % kLanes;
    const int rsub = lane / kLanes;
    const Pieces pc = pieces<D>(p, sub);

    if (blockIdx.x >= kv_ctas) {
        // ---- queries: kQueryPasses * kRows rows a warp, their loads in flight together ------------------------------
        const unsigned item = (blockIdx.x - kv_ctas) * kAppWarps + warp;  // fewer than 2^31
        uint4 va[kQueryPasses], vb[kQueryPasses];
        if (head_blocks > 0) {  // whole blocks of one token's heads: its range, position and angles are taken once
            const unsigned token = item / static_cast<unsigned>(head_blocks);
            const int h0 = static_cast<int>(item - token * head_blocks) * (kQueryPasses * kRows) + rsub;
            const int b = static_cast<int>(token / static_cast<unsigned>(p.n_new));
            if (b >= p.B) return;
            const int j = static_cast<int>(token - static_cast<unsigned>(b) * p.n_new);
            int tb, te;
            if (!token_range(p, b, tb, te, false) || j >= te - tb) return;
            const int pos = position(p, b, j, tb + j);
            if (pos < 0) {
                if (lane == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
                return;
            }
            const kvmm_bf16* src = p.q.data + b * p.q.batch_stride + j * p.q.token_stride;
            uint4* dst = reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(token) * p.Hq + h0) * D);
#pragma unroll
            for (int k = 0; k < kQueryPasses; ++k) {
                const uint4* row = reinterpret_cast<const uint4*>(src + (h0 + k * kRows) * p.q.head_stride);
                va[k] = row[pc.a];
                vb[k] = row[pc.b];
            }
            Angles g{};
            if (pc.turns) g = angles(p, pos, pc);
#pragma unroll
            for (int k = 0; k < kQueryPasses; ++k) {
                if (pc.turns) turn_row(p, g, va[k], vb[k]);
                dst[k * kRows * (D / 8) + pc.a] = va[k];
                dst[k * kRows * (D / 8) + pc.b] = vb[k];
            }
            return;
        }
        // other head counts: consecutive (batch, token, head) rows, each with its own range, position and angles
        const unsigned rows = static_cast<unsigned>(p.B) * p.n_new * p.Hq;  // fewer than 2^32
        const unsigned row0 = item * (kQueryPasses * kRows) + rsub;
        int b[kQueryPasses], j[kQueryPasses], h[kQueryPasses], tb[kQueryPasses], te[kQueryPasses];
#pragma unroll
        for (int k = 0; k < kQueryPasses; ++k) {
            const unsigned row = min(row0 + k * kRows, rows - 1);
            const unsigned token = row / static_cast<unsigned>(p.Hq);
            h[k] = static_cast<int>(row - token * p.Hq);
            b[k] = static_cast<int>(token / static_cast<unsigned>(p.n_new));
            j[k] = static_cast<int>(token - static_cast<unsigned>(b[k]) * p.n_new);
            tb[k] = p.tok_begin[b[k]];
            te[k] = p.tok_end[b[k]];
        }
        int at[kQueryPasses];  // its position, -1: no row
#pragma unroll
        for (int k = 0; k < kQueryPasses; ++k) {
            const int n = token_count(p, tb[k], te[k]);
            at[k] = -1;
            if (row0 + k * kRows < rows && j[k] < n) {
                at[k] = position(p, b[k], j[k], tb[k] + j[k]);
                if (at[k] < 0 && sub == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
            }
        }
#pragma unroll
        for (int k = 0; k < kQueryPasses; ++k)
            if (at[k] >= 0) {
                const uint4* row = reinterpret_cast<const uint4*>(p.q.data + b[k] * p.q.batch_stride +
                                                                  j[k] * p.q.token_stride + h[k] * p.q.head_stride);
                va[k] = row[pc.a];
                vb[k] = row[pc.b];
            }
#pragma unroll
        for (int k = 0; k < kQueryPasses; ++k)
            if (at[k] >= 0) {
                if (pc.turns) turn_row(p, angles(p, at[k], pc), va[k], vb[k]);
                uint4* dst = reinterpret_cast<uint4*>(p.q_out + static_cast<size_t>(row0 + k * kRows) * D);
                dst[pc.a] = va[k];
                dst[pc.b] = vb[k];
            }
        return;
    }

    // ---- keys and values: one page of one (batch, KV head) a warp, the heads of a page side by side -----------
    const unsigned item = blockIdx.x * kAppWarps + warp;  // fewer than 2^31
    const unsigned pages = item / static_cast<unsigned>(p.Hkv);
    const int h = static_cast<int>(item - pages * p.Hkv);
    const int b = static_cast<int>(pages / static_cast<unsigned>(page_slots));
    if (b >= p.B) return;
    const int slot = static_cast<int>(pages - static_cast<unsigned>(b) * page_slots);
    int tb, te;
    if (!token_range(p, b, tb, te, slot == 0 && h == 0 && lane == 0)) return;
    const int page = tb / T + slot;
    const int first = page * T;
    if (first >= te) return;
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer) * p.Hkv + h;
    const int32_t phys = p.block_table[unit * p.Pmax + page];
    if (phys < 0 || phys >= p.n_phys) {
        if (lane == 0) report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    // rows of the page this call writes (`fresh`), and those that stay and count for its MinMax (`held`); lane r < T
    // has the position of row r
    const int r0 = max(tb - first, 0), r1 = min(te - first, T);
    int pos = -1;
    if (lane >= r0 && lane < r1) {
        pos = position(p, b, first + lane - tb, first + lane);
        if (pos < 0 && h == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
    }
    const unsigned fresh = __ballot_sync(kFullMask, pos >= 0);
    const unsigned held = p.meta != nullptr ? ((r1 < 32 ? (1u << r1) : 0u) - 1u) & ~fresh : 0u;
    const kvmm_bf16* k_src = p.k.data + b * p.k.batch_stride + h * p.k.head_stride + (first - tb) * p.k.token_stride;
    const kvmm_bf16* v_src = p.v.data + b * p.v.batch_stride + h * p.v.head_stride + (first - tb) * p.v.token_stride;
    uint8_t* page4 = KV4 ? p.kv4_pool + static_cast<size_t>(phys) * Page::kBytes : nullptr;
    kvmm_bf16* kpage = KV4 ? nullptr : p.k_pool + static_cast<size_t>(phys) * T * D;
    kvmm_bf16* vpage = KV4 ? nullptr : p.v_pool + static_cast<size_t>(phys) * T * D;
    constexpr unsigned kBatchRows = kRows * kBatch == 32 ? ~0u : (1u << (kRows * kBatch)) - 1u;

    // Infinite values of 4-bit rows are looked for once a page, over the largest magnitudes that are there anyway, and
    // the page's rows are then done again with limits (two chunks of 8K: 64.4 us; limits on every channel 65.8, a vote
    // a row 65.2, without either 64.7).
    Bounds ba, bb;
    float most = 0.f;
    auto rows = [&](auto limit) {
        ba.clear();
        bb.clear();
#pragma unroll 1
        for (int i0 = 0; i0 < T; i0 += kRows * kBatch) {
            const unsigned here = kBatchRows << i0;
            if ((held & here) != 0u) {
                uint4 va[kBatch], vb[kBatch];
                if (KV4) {
                    uint32_t ca[kBatch], cb[kBatch], sa[kBatch], sb[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int r = i0 + i * kRows + rsub;
                        const uint32_t* cd = reinterpret_cast<const uint32_t*>(page4 + r * Page::kRow);
                        const uint8_t* sc = page4 + Page::kKeyScales + r * Page::kGroups;
                        ca[i] = cd[pc.a], cb[i] = cd[pc.b], sa[i] = sc[pc.a >> 1], sb[i] = sc[pc.b >> 1];
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) va[i] = held8(ca[i], sa[i]), vb[i] = held8(cb[i], sb[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const uint4* src = reinterpret_cast<const uint4*>(kpage + (i0 + i * kRows + rsub) * D);
                        va[i] = src[pc.a];
                        vb[i] = src[pc.b];
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (held >> (i0 + i * kRows + rsub) & 1u) {
                        ba.add(va[i]);
                        bb.add(vb[i]);
                    }
            }
            if ((fresh & here) == 0u) continue;
            uint4 va[kBatch], vb[kBatch], wa[KV4 ? kBatch : 1], wb[KV4 ? kBatch : 1];
            Angles g[kBatch];
            bool mine[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = i0 + i * kRows + rsub;
                const int at = __shfl_sync(kFullMask, pos, r);
                mine[i] = at >= 0;
                va[i] = vb[i] = make_uint4(0u, 0u, 0u, 0u);
                if (KV4) wa[i] = wb[i] = va[i];
                if (mine[i]) {
                    const uint4* src = reinterpret_cast<const uint4*>(k_src + r * p.k.token_stride);
                    va[i] = src[pc.a];
                    vb[i] = src[pc.b];
                    if (KV4) {
                        src = reinterpret_cast<const uint4*>(v_src + r * p.v.token_stride);
                        wa[i] = src[pc.a];
                        wb[i] = src[pc.b];
                    }
                    if (pc.turns) g[i] = angles(p, at, pc);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = i0 + i * kRows + rsub;
                float a[8], c[8];
                unpack8(va[i], a);
                unpack8(vb[i], c);
                if (mine[i] && pc.turns) rotate(p, g[i], a, c);
                if (KV4) {
                    uint32_t ca, cb, sa, sb;
                    hold4<decltype(limit)::value>(a, c, p.k_inv, ca, cb, sa, sb, most);
                    float x[8], y[8];
                    unpack8(wa[i], x);
                    unpack8(wb[i], y);
                    uint32_t da, db, ta, tb4;
                    hold4<decltype(limit)::value>(x, y, p.v_inv, da, db, ta, tb4, most);
                    if (mine[i]) {
                        uint32_t* cd = reinterpret_cast<uint32_t*>(page4 + r * Page::kRow);
                        cd[pc.a] = ca;
                        cd[pc.b] = cb;
                        cd = reinterpret_cast<uint32_t*>(page4 + Page::kValues + r * Page::kRow);
                        cd[pc.a] = da;
                        cd[pc.b] = db;
                        if ((sub & 1) == 0) {
                            uint8_t* sc = page4 + Page::kKeyScales + r * Page::kGroups;
                            sc[pc.a >> 1] = static_cast<uint8_t>(sa);
                            sc[pc.b >> 1] = static_cast<uint8_t>(sb);
                            sc = page4 + Page::kValueScales + r * Page::kGroups;
                            sc[pc.a >> 1] = static_cast<uint8_t>(ta);
                            sc[pc.b >> 1] = static_cast<uint8_t>(tb4);
                        }
                        if (p.meta != nullptr) {
                            ba.add(held8(ca, sa));
                            bb.add(held8(cb, sb));
                        }
                    }
                } else if (mine[i]) {
                    if (pc.turns) {
                        va[i] = pack8(a);
                        vb[i] = pack8(c);
                    }
                    uint4* dst = reinterpret_cast<uint4*>(kpage + r * D);
                    dst[pc.a] = va[i];
                    dst[pc.b] = vb[i];
                    ba.add(va[i]);
                    bb.add(vb[i]);
                }
            }
        }
    };
    rows(std::false_type{});
    if constexpr (KV4) {
        if (__any_sync(kFullMask, most > FLT_MAX)) rows(std::true_type{});
    }
    if (p.meta != nullptr) {
#pragma unroll
        for (int off = kLanes; off < 32; off <<= 1) {
            ba.across(off);
            bb.across(off);
        }
        if (rsub == 0) {
            kvmm_bf16* m = p.meta + (unit * p.Pmax + page) * 2 * D;
            ba.store(m, D, pc.a);
            bb.store(m, D, pc.b);
        }
    }

    if (!KV4) {
        // values go dimension-major: a lane moves two channels of 16 tokens (coalesced 4-byte loads of the rows,
        // 32 bytes of one channel's tokens a store)
#pragma unroll 1
        for (int t0 = 0; t0 < T; t0 += 16) {
            const unsigned have = fresh >> t0 & 0xffffu;
            if (have == 0u) continue;
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += 64) {
                const int d = d0 + 2 * lane;
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (have >> i & 1u) w[i] = *reinterpret_cast<const uint32_t*>(v_src + (t0 + i) * p.v.token_stride + d);
                kvmm_bf16* c0 = vpage + d * T + t0;
                kvmm_bf16* c1 = c0 + T;
                if (have == 0xffffu) {
                    uint32_t a[8], c[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] = prmt(w[2 * i], w[2 * i + 1], 0x5410);
                        c[i] = prmt(w[2 * i], w[2 * i + 1], 0x7632);
                    }
                    reinterpret_cast<uint4*>(c0)[0] = make_uint4(a[0], a[1], a[2], a[3]);
                    reinterpret_cast<uint4*>(c0)[1] = make_uint4(a[4], a[5], a[6], a[7]);
                    reinterpret_cast<uint4*>(c1)[0] = make_uint4(c[0], c[1], c[2], c[3]);
                    reinterpret_cast<uint4*>(c1)[1] = make_uint4(c[4], c[5], c[6], c[7]);
                } else if (__popc(have) > 2) {
                    // some of the 16 tokens: put among those that are there and stored back whole (2-byte stores of 31
                    // of a page's 32 tokens took ten times as long as the whole page)
                    uint32_t a[8], c[8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 x = reinterpret_cast<const uint4*>(c0)[i], y = reinterpret_cast<const uint4*>(c1)[i];
                        a[4 * i] = x.x, a[4 * i + 1] = x.y, a[4 * i + 2] = x.z, a[4 * i + 3] = x.w;
                        c[4 * i] = y.x, c[4 * i + 1] = y.y, c[4 * i + 2] = y.z, c[4 * i + 3] = y.w;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (have >> i & 1u) {  // (i even: the low half of the word)
                            a[i / 2] = i % 2 ? prmt(a[i / 2], w[i], 0x5410) : prmt(a[i / 2], w[i], 0x3254);
                            c[i / 2] = i % 2 ? prmt(c[i / 2], w[i], 0x7610) : prmt(c[i / 2], w[i], 0x3276);
                        }
                    reinterpret_cast<uint4*>(c0)[0] = make_uint4(a[0], a[1], a[2], a[3]);
                    reinterpret_cast<uint4*>(c0)[1] = make_uint4(a[4], a[5], a[6], a[7]);
                    reinterpret_cast<uint4*>(c1)[0] = make_uint4(c[0], c[1], c[2], c[3]);
                    reinterpret_cast<uint4*>(c1)[1] = make_uint4(c[4], c[5], c[6], c[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (have >> i & 1u) {
                            c0[i] = static_cast<kvmm_bf16>(w[i] & 0xffffu);
                            c1[i] = static_cast<kvmm_bf16>(w[i] >> 16);
                        }
                }
            }
        }
    }
}

template <int D, int T>
cudaError_t launch(const AppendParams& p, cudaStream_t stream)
{
    // pages one batch entry can reach, and the warps that move them and the query rows
    const long long span = (static_cast<long long>(p.n_new) + T - 1) / T + 1;
    const int slots = static_cast<int>(span < p.Pmax ? span : p.Pmax);
    const long long items = static_cast<long long>(p.B) * slots * p.Hkv;
    const long long kv_ctas = (items + kAppWarps - 1) / kAppWarps;
    // queries: whole blocks of a token's heads where these divide them, else rows of the list
    constexpr int kHeads = kQueryPasses * 32 / (D / 16);
    const int head_blocks = p.Hq % kHeads == 0 ? p.Hq / kHeads : 0;
    const long long rows = p.q.data ? static_cast<long long>(p.B) * p.n_new * p.Hq : 0;
    const long long q_items = (rows + kHeads - 1) / kHeads;
    if (rows > 0xffffffffll - kHeads) return cudaErrorInvalidConfiguration;  // (terabytes of rows)
    const long long ctas = kv_ctas + (q_items + kAppWarps - 1) / kAppWarps;
    if (ctas > 0x7fffffffll / kAppWarps) return cudaErrorInvalidConfiguration;  // (terabytes of rows)
    void (*kernel)(AppendParams, int, unsigned, int) =
        p.kv4_pool ? append_rope_kernel<D, T, true> : append_rope_kernel<D, T, false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAppWarps * 32), 0, stream, p, slots,
                      static_cast<unsigned>(kv_ctas), head_blocks);
}

}  // namespace

cudaError_t launch_append_rope(const AppendParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
