// kv4_gather.cu -- tokens of the 4-bit cache back as bf16 rows.
//
// value = code * scale * factor: the product of code and scale is exact in
// fp16, so one fp32 multiplication and one rounding to bf16 follow it.
// One warp takes one page of one (batch, KV head): a lane turns eight codes (4
// bytes) and their scale into 16 bytes of a row, so both sides of the copy are
// coalesced.  Bound by the bytes written (2 of them for 0.56 read): 72K tokens
// of 8 heads (265 MB) take 45.8 us, 0.85 of a copy's rate; more or fewer loads
// in flight, both sides' loads first, 4 or 16 warps a CTA and streaming stores
// were all within 1% of it.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace kvmm {
namespace {

constexpr int kGatWarps = 8;

__device__ __forceinline__ uint4 values8(uint32_t code, uint32_t scale, float factor)
{
    const uint32_t s = e4m3x2_to_half2(scale | (scale << 8));
    const uint32_t h[4] = {half2_mul(e2m1x2_to_half2<0>(code), s), half2_mul(e2m1x2_to_half2<1>(code), s),
                           half2_mul(e2m1x2_to_half2<2>(code), s), half2_mul(e2m1x2_to_half2<3>(code), s)};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(__fmul_rn(half_lo(h[i]), factor), __fmul_rn(half_hi(h[i]), factor));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, int T>
__global__ void __launch_bounds__(kGatWarps * 32) kv4_gather_kernel(const GatherParams p, int page_slots)
{
    using Page = Kv4Page<D, T>;
    constexpr int kLanes = D / 8;       // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows a warp moves at once
    constexpr int kBatch = T / kRows < 8 ? T / kRows : 8;  // loads in flight a lane
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * kGatWarps + (threadIdx.x >> 5);  // fewer than 2^31
    const unsigned pages = item / static_cast<unsigned>(p.Hkv);
    const int h = static_cast<int>(item - pages * p.Hkv);
    const int b = static_cast<int>(pages / static_cast<unsigned>(page_slots));
    if (b >= p.B) return;
    const int slot = static_cast<int>(pages - static_cast<unsigned>(b) * page_slots);
    const bool tell = slot == 0 && h == 0 && lane == 0;
    const int cap = p.Pmax * T;
    int tb = p.tok_begin ? p.tok_begin[b] : 0, te = p.tok_end[b];
    if (tb < 0 || te < tb || te > cap) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        tb = max(tb, 0);
        te = min(max(te, tb), cap);
    }
    if (te - tb > p.n_rows) {
        if (tell) report(p.err, KVMM_ERR_OUT_OF_RANGE);
        te = tb + p.n_rows;
    }
    const int page = tb / T + slot;
    if (te <= tb || page * T >= te) return;
    const size_t unit = (static_cast<size_t>(b) * p.L + p.layer) * p.Hkv + h;
    const int32_t phys = p.block_table[unit * p.Pmax + page];
    if (phys < 0 || phys >= p.n_phys) {
        if (lane == 0) report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
        return;
    }
    const int r0 = max(tb - page * T, 0), r1 = min(te - page * T, T);
    const int piece = lane % kLanes, rsub = lane / kLanes;
    const uint8_t* src = p.kv4_pool + static_cast<size_t>(phys) * Page::kBytes;
    // row 0 of the page among the rows asked for (may lie before the first: only rows r0 .. r1 - 1 are written)
    const int64_t row0 = static_cast<int64_t>(b) * p.n_rows + (page * T - tb);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        kvmm_bf16* out = side ? p.v_out : p.k_out;
        if (out == nullptr) continue;
        const uint8_t* codes = src + (side ? Page::kValues : 0);
        const uint8_t* scales = src + (side ? Page::kValueScales : Page::kKeyScales);
        const float factor = side ? p.v_scale : p.k_scale;
#pragma unroll
        for (int i0 = 0; i0 < T / kRows; i0 += kBatch) {
            uint32_t cd[kBatch], sc[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = (i0 + i) * kRows + rsub;
                cd[i] = reinterpret_cast<const uint32_t*>(codes + r * Page::kRow)[piece];
                sc[i] = scales[r * Page::kGroups + (piece >> 1)];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = (i0 + i) * kRows + rsub;
                if (r >= r0 && r < r1)
                    reinterpret_cast<uint4*>(out + ((row0 + r) * p.Hkv + h) * D)[piece] = values8(cd[i], sc[i], factor);
            }
        }
    }
}

template <int D, int T>
cudaError_t launch(const GatherParams& p, cudaStream_t stream)
{
    const long long span = (static_cast<long long>(p.n_rows) + T - 1) / T + 1;  // pages one range can reach
    const int slots = static_cast<int>(span < p.Pmax ? span : p.Pmax);
    const long long ctas = (static_cast<long long>(p.B) * slots * p.Hkv + kGatWarps - 1) / kGatWarps;
    if (ctas > 0x7fffffffll / kGatWarps) return cudaErrorInvalidConfiguration;  // (terabytes of rows)
    return launch_pdl(kv4_gather_kernel<D, T>, dim3(static_cast<unsigned>(ctas)), dim3(kGatWarps * 32), 0, stream, p,
                      slots);
}

}  // namespace

cudaError_t launch_kv4_gather(const GatherParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
