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
// alone) by the same loads as the new ones.  Further warps rotate the query
// rows.  The pass is bound by the bytes it moves for prompts and by the chain
// of dependent loads (range, table entry, rows) for single tokens.
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

// rotate a lane's two pieces (channels 8*ca.. and 8*cb..) by table row `pos`
__device__ __forceinline__ void rotate(const AppendParams& p, int pos, int ca, int cb, float (&a)[8], float (&b)[8])
{
    const float* cs = p.rope.table + static_cast<size_t>(pos) * p.rope.dim;
    const float* sn = cs + p.rope.dim / 2;
    if (p.rope.interleaved) {  // pairs inside a piece: angles 4c .. 4c+3
        const float4 c0 = *reinterpret_cast<const float4*>(cs + 4 * ca), s0 = *reinterpret_cast<const float4*>(sn + 4 * ca);
        const float4 c1 = *reinterpret_cast<const float4*>(cs + 4 * cb), s1 = *reinterpret_cast<const float4*>(sn + 4 * cb);
        turn(a[0], a[1], c0.x, s0.x);
        turn(a[2], a[3], c0.y, s0.y);
        turn(a[4], a[5], c0.z, s0.z);
        turn(a[6], a[7], c0.w, s0.w);
        turn(b[0], b[1], c1.x, s1.x);
        turn(b[2], b[3], c1.y, s1.y);
        turn(b[4], b[5], c1.z, s1.z);
        turn(b[6], b[7], c1.w, s1.w);
    } else {  // channel i with i + dim/2: angles 8*ca .. 8*ca+7
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 c = reinterpret_cast<const float4*>(cs + 8 * ca)[i];
            const float4 s = reinterpret_cast<const float4*>(sn + 8 * ca)[i];
            turn(a[4 * i], b[4 * i], c.x, s.x);
            turn(a[4 * i + 1], b[4 * i + 1], c.y, s.y);
            turn(a[4 * i + 2], b[4 * i + 2], c.z, s.z);
            turn(a[4 * i + 3], b[4 * i + 3], c.w, s.w);
        }
    }
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

// Hold a lane's two pieces in 4 bits: codes (eight nibbles a piece) and the
// scales' bytes; `a`, `b` become code * scale.  Every lane of the warp calls.
__device__ __forceinline__ void hold4(float (&a)[8], float (&b)[8], float inv, uint32_t& code_a, uint32_t& code_b,
                                      uint32_t& scale_a, uint32_t& scale_b)
{
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = __fmul_rn(a[i], inv);
        b[i] = __fmul_rn(b[i], inv);
        ma = fmaxf(ma, fabsf(a[i]));
        mb = fmaxf(mb, fabsf(b[i]));
    }
    ma = fmaxf(ma, __shfl_xor_sync(kFullMask, ma, 1));  // the other eight channels of the scale
    mb = fmaxf(mb, __shfl_xor_sync(kFullMask, mb, 1));
    scale_a = float_to_e4m3(__fdiv_rn(ma, 6.f));
    scale_b = float_to_e4m3(__fdiv_rn(mb, 6.f));
    const uint32_t s2 = e4m3x2_to_half2(scale_a | (scale_b << 8));
    const float sa = half_lo(s2), sb = half_hi(s2);
    code_a = code_b = 0u;
    // A quotient is rounded to fp32, then to e2m1.  y has 24 significant bits and the scale 4, so a quotient
    // that is not a border of e2m1 does not round to one: the code is the nearest to the true quotient.
    if (scale_a != 0u) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code_a |= float2_to_e2m1x2(__fdiv_rn(a[2 * i], sa), __fdiv_rn(a[2 * i + 1], sa)) << (8 * i);
    }
    if (scale_b != 0u) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code_b |= float2_to_e2m1x2(__fdiv_rn(b[2 * i], sb), __fdiv_rn(b[2 * i + 1], sb)) << (8 * i);
    }
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

template <int D, int T, bool KV4>
__global__ void __launch_bounds__(kAppWarps * 32) append_rope_kernel(const AppendParams p, int page_slots,
                                                                     unsigned kv_ctas, int q_passes)
{
    using Page = Kv4Page<D, T>;
    constexpr int kLanes = D / 16;        // lanes of a row
    constexpr int kRows = 32 / kLanes;    // rows a warp moves at once
    pdl_wait_then_release();  // the pools, table and metadata may be in use by the previous kernel
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int sub = lane % kLanes;
    const int rsub = lane / kLanes;
    const Pieces pc = pieces<D>(p, sub);

    if (blockIdx.x >= kv_ctas) {
        // ---- query rows: q_passes * kRows consecutive (batch, token, head) rows a warp --------------------
        const int64_t rows = static_cast<int64_t>(p.B) * p.n_new * p.Hq;
        const int64_t first = (static_cast<int64_t>(blockIdx.x - kv_ctas) * kAppWarps + warp) * q_passes * kRows;
        for (int k = 0; k < q_passes; ++k) {
            const int64_t row = first + k * kRows + rsub;
            if (row >= rows) continue;
            const int64_t bt = row / p.Hq;
            const int h = static_cast<int>(row - bt * p.Hq);
            const int b = static_cast<int>(bt / p.n_new);
            const int j = static_cast<int>(bt - static_cast<int64_t>(b) * p.n_new);
            int tb, te;
            if (!token_range(p, b, tb, te, false) || j >= te - tb) continue;
            const int pos = position(p, b, j, tb + j);
            if (pos < 0) {
                if (sub == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
                continue;
            }
            const uint4* src = reinterpret_cast<const uint4*>(p.q.data + b * p.q.batch_stride +
                                                              j * p.q.token_stride + h * p.q.head_stride);
            uint4* dst = reinterpret_cast<uint4*>(p.q_out + row * D);
            uint4 va = src[pc.a], vb = src[pc.b];
            if (pc.turns) {
                float a[8], c[8];
                unpack8(va, a);
                unpack8(vb, c);
                rotate(p, pos, pc.a, pc.b, a, c);
                va = pack8(a);
                vb = pack8(c);
            }
            dst[pc.a] = va;
            dst[pc.b] = vb;
        }
        return;
    }

    // ---- keys and values: one page of one (batch, KV head) a warp, the heads of a page side by side -----------
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kAppWarps + warp;
    const int64_t pages = item / p.Hkv;
    const int h = static_cast<int>(item - pages * p.Hkv);
    const int b = static_cast<int>(pages / page_slots);
    if (b >= p.B) return;
    const int slot = static_cast<int>(pages - static_cast<int64_t>(b) * page_slots);
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
    const int r0 = max(tb - first, 0);      // new rows of the page: [r0, r1); rows before r0 are there already
    const int r1 = min(te - first, T);
    const kvmm_bf16* k_src = p.k.data + b * p.k.batch_stride + h * p.k.head_stride;
    const kvmm_bf16* v_src = p.v.data + b * p.v.batch_stride + h * p.v.head_stride;
    uint8_t* page4 = KV4 ? p.kv4_pool + static_cast<size_t>(phys) * Page::kBytes : nullptr;
    kvmm_bf16* kpage = KV4 ? nullptr : p.k_pool + static_cast<size_t>(phys) * T * D;
    kvmm_bf16* vpage = KV4 ? nullptr : p.v_pool + static_cast<size_t>(phys) * T * D;

    Bounds ba, bb;
    ba.clear();
    bb.clear();
#pragma unroll 4
    for (int i = 0; i < T / kRows; ++i) {
        const int r = i * kRows + rsub;
        const int j = first + r - tb;  // its row among the new ones
        int pos = -1;
        if (r >= r0 && r < r1) {
            pos = position(p, b, j, first + r);
            if (pos < 0 && sub == 0 && h == 0) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        }
        const bool fresh = pos >= 0;
        const bool held = !fresh && r < r1 && p.meta != nullptr;  // read back for the MinMax
        uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
        if (fresh) {
            const uint4* src = reinterpret_cast<const uint4*>(k_src + j * p.k.token_stride);
            va = src[pc.a];
            vb = src[pc.b];
        } else if (held) {
            if (KV4) {
                const uint8_t* sc = page4 + Page::kKeyScales + r * Page::kGroups;
                const uint32_t* cd = reinterpret_cast<const uint32_t*>(page4 + r * Page::kRow);
                va = held8(cd[pc.a], sc[pc.a >> 1]);
                vb = held8(cd[pc.b], sc[pc.b >> 1]);
            } else {
                const uint4* src = reinterpret_cast<const uint4*>(kpage + static_cast<size_t>(r) * D);
                va = src[pc.a];
                vb = src[pc.b];
            }
        }
        if (KV4) {
            float a[8], c[8];
            unpack8(va, a);
            unpack8(vb, c);
            if (fresh && pc.turns) rotate(p, pos, pc.a, pc.b, a, c);
            uint32_t ca, cb, sa, sb;
            hold4(a, c, p.k_inv, ca, cb, sa, sb);
            if (fresh) {
                uint32_t* cd = reinterpret_cast<uint32_t*>(page4 + r * Page::kRow);
                cd[pc.a] = ca;
                cd[pc.b] = cb;
                if ((sub & 1) == 0) {
                    uint8_t* sc = page4 + Page::kKeyScales + r * Page::kGroups;
                    sc[pc.a >> 1] = static_cast<uint8_t>(sa);
                    sc[pc.b >> 1] = static_cast<uint8_t>(sb);
                }
                va = held8(ca, sa);
                vb = held8(cb, sb);
            }
        } else if (fresh) {
            if (pc.turns) {
                float a[8], c[8];
                unpack8(va, a);
                unpack8(vb, c);
                rotate(p, pos, pc.a, pc.b, a, c);
                va = pack8(a);
                vb = pack8(c);
            }
            uint4* dst = reinterpret_cast<uint4*>(kpage + static_cast<size_t>(r) * D);
            dst[pc.a] = va;
            dst[pc.b] = vb;
        }
        if (fresh || held) {
            ba.add(va);
            bb.add(vb);
        }
        if (KV4) {
            uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
            if (fresh) {
                const uint4* src = reinterpret_cast<const uint4*>(v_src + j * p.v.token_stride);
                wa = src[pc.a];
                wb = src[pc.b];
            }
            float a[8], c[8];
            unpack8(wa, a);
            unpack8(wb, c);
            uint32_t ca, cb, sa, sb;
            hold4(a, c, p.v_inv, ca, cb, sa, sb);
            if (fresh) {
                uint32_t* cd = reinterpret_cast<uint32_t*>(page4 + Page::kValues + r * Page::kRow);
                cd[pc.a] = ca;
                cd[pc.b] = cb;
                if ((sub & 1) == 0) {
                    uint8_t* sc = page4 + Page::kValueScales + r * Page::kGroups;
                    sc[pc.a >> 1] = static_cast<uint8_t>(sa);
                    sc[pc.b >> 1] = static_cast<uint8_t>(sb);
                }
            }
        }
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
#pragma unroll
        for (int t0 = 0; t0 < T; t0 += 16) {
            if (t0 >= r1 || t0 + 16 <= r0) continue;
            const bool whole = t0 >= r0 && t0 + 16 <= r1;
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += 64) {
                const int d = d0 + 2 * lane;
                uint32_t w[16];
                unsigned have = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = t0 + i, j = first + r - tb;
                    w[i] = 0u;
                    if (r >= r0 && r < r1 && position(p, b, j, first + r) >= 0) {
                        w[i] = *reinterpret_cast<const uint32_t*>(v_src + j * p.v.token_stride + d);
                        have |= 1u << i;
                    }
                }
                kvmm_bf16* c0 = vpage + static_cast<size_t>(d) * T + t0;
                kvmm_bf16* c1 = c0 + T;
                if (whole && have == 0xffffu) {
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
    constexpr int kRows = 32 / (D / 16);
    const long long rows = p.q.data ? static_cast<long long>(p.B) * p.n_new * p.Hq : 0;
    const int passes = rows >= 65536 ? 4 : 1;
    const long long per_cta = static_cast<long long>(kAppWarps) * kRows * passes;
    const long long ctas = kv_ctas + (rows + per_cta - 1) / per_cta;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    void (*kernel)(AppendParams, int, unsigned, int) =
        p.kv4_pool ? append_rope_kernel<D, T, true> : append_rope_kernel<D, T, false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAppWarps * 32), 0, stream, p, slots,
                      static_cast<unsigned>(kv_ctas), passes);
}

}  // namespace

cudaError_t launch_append_rope(const AppendParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
