// kv4_attn.cu -- decode attention over the 4-bit cache: selected pages, or
// every page of a sequence.
//
// For the G query heads of a KV head, over the tokens of the unit's pages,
//   z = q . k,  out = sum_t 2^(z_t - m) v_t / sum_t 2^(z_t - m)
// in one pass with a running reference m (sm_scale, k_scale and log2(e) are one
// factor on z; v_scale is applied to the result).
//
// Work.  With no more units than SMs, and with selections or short sequences
// (kShortTiles), each unit has a cluster of CTAs (as many as all run at once),
// which share its places (selections: Kmax) or its sequence's pages and merge
// their parts through distributed shared memory.  Else the pages of all units
// form one list (with selections, Kmax places a unit) and CTA c of the N
// launched, one for each SM, takes the c-th of N equal pieces of it, whatever
// the sequences' lengths, so there is one wave without a tail.
// A step is two pages of 16 tokens or one of 32.  Sixteen warps take a cluster
// CTA's steps in turn; of an even piece each takes a run, so that it meets few
// units (832 units of up to 764 tokens: 46.7 us in turn, with every unit merged
// from all sixteen, against 28.9 when runs came; 29.9 now).  Each warp's steps pass through a ring of its own,
// filled by one bulk copy a page (with the L2 policy of data read once), and run
// ahead across units.  What a warp has of a unit that is not its alone goes to
// shared memory, and once a CTA the parts are joined.  A unit that lies in one
// CTA is then written out; the parts of the others (two a CTA at most: its first
// and its last unit) go to the workspace, and the CTA that stores a unit's last
// part, as a counter tells it, combines them.
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
//
// Bound and measured (one GB300, us a launch in a graph of launches over three
// inputs; the bytes are what the tokens hold, against the 6.78 TB/s of a copy).
//   every page, one 128K sequence, 8 KV heads (151 MB)          35.6  0.63
//   every page, 32 ragged sequences up to 16K tokens (449 MB)   85.7  0.77
//   128 selected pages a head, 32K context, batch 8 (19 MB)     10.9  0.26
//   64 pages of 32 tokens, five heads a KV head, batch 16 (36 MB) 13.7  0.39
// Inside the long calls a tile takes 99 clocks an SM at 128K, the rate of the
// memory.  Of the launch's 338 instructions a tile (all of them over all tiles)
// 237 are the tile's own (68 conversions, 64 products with scales, 16 MMAs).
// What is left is latency (clock stamps at 128K, of a state of 36.2 us): lengths,
// table and first pages 4.0 us, warps that end up to 2.9 us apart, the joins of
// warps, then of CTAs 6.6 us.  Short calls are that and the tiles' 95 clocks, on
// the 128 SMs that whole clusters fill.
// Measured and not kept: a second launch for the merge (6 us of 20 at 32K), a
// producer warp for all rings (the copies of one warp's lanes go out one after
// another, 70 clocks each: 111 us against 97 for the ragged batch then), 8 or 12
// warps with longer rings (124 and 112 against 106 then), runs joined with all
// their parts' reads unrolled (34.0 us against 28.9 for the 832 units) or a
// cluster's by that short loop (12.2 against 10.4 for the selections).
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace kvmm {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kShortTiles = 256;               // over every page: most 16-token tiles a CTA of a unit's cluster has
constexpr int kStep = 32;                      // tokens of a step: two pages of 16, or one of 32
constexpr uint64_t kWaitNs = 1000000000ull;    // far beyond any legitimate wait
__host__ __device__ constexpr int ring_depth(int D) { return D == 64 ? 4 : 2; }  // steps in flight a warp
__host__ __device__ constexpr int step_bytes(int D) { return kStep * (D + D / 8); }

struct Shared {
    uint64_t full[kWarps][4];  // a step has landed
    int2 meta[kWarps][4];      // per tile of the step: unit * 64 + valid tokens
    float m[2 * kWarps][8];    // each part's reference per head
    float l[2 * kWarps][8];    // ... and sum
    int unit[2 * kWarps];      // ... and unit, -1: none
    float weight[2 * kWarps][8];  // the parts there are, in order: their weights
    int at[2 * kWarps];           // ... and places
    int scan[kWarps];
    int total;                 // pages of the list
    int span[2][2];            // units that several CTAs share: the first CTA, and, for the one that merges, how many
    float recv[8 * 128 + kKv4MaxCluster];  // received: every CTA's partial of this CTA's slice of the outputs
    float rstat[kKv4MaxCluster][16];       // received: (reference, sum) per head of every CTA of the cluster
};

// A warp's part of a unit: a row of D + 8 floats a head, the D/8 channels of a row group one float apart from the next
// group's (the lanes of a store then fall on different banks).  A warp has two at most: part 2 * warp, of the unit that
// began before its piece and ends in it, has a place of its own; part 2 * warp + 1, of the unit its piece ends in, goes
// where its ring was.
__host__ __device__ constexpr int part_row(int D) { return D + 8; }
static_assert(8 * part_row(128) * sizeof(float) <= ring_depth(128) * step_bytes(128) &&
              8 * part_row(64) * sizeof(float) <= ring_depth(64) * step_bytes(64), "a part fits the ring");
// dynamic shared memory: [rings][parts][first pages and page counts of the batch]
__host__ __device__ constexpr size_t part_offset(int D) { return size_t(kWarps) * ring_depth(D) * step_bytes(D); }
__host__ __device__ inline size_t list_offset(int D, int G)
{
    return part_offset(D) + size_t(kWarps) * G * part_row(D) * sizeof(float);
}
inline size_t smem_bytes(int D, int G, int nb) { return list_offset(D, G) + size_t(2 * nb + 1) * sizeof(int); }

// o += c for the four accumulators of a tile, two additions an instruction
__device__ __forceinline__ void add4(float (&o)[4], const float (&c)[4])
{
#pragma unroll
    for (int k = 0; k < 4; k += 2)
        asm("{.reg .b64 p, q; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %3}; add.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p;}"
            : "+f"(o[k]), "+f"(o[k + 1])
            : "f"(c[k]), "f"(c[k + 1]));
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// `total` pages dealt to n CTAs: CTA c's piece starts at floor(c * total / n), so that units of one length of which
// each fills the same number of CTAs begin where a piece does
struct Pieces {
    int total, n, each, more;
    __device__ __forceinline__ Pieces(int total_, int n_) : total(total_), n(n_), each(total_ / n_), more(total_ % n_) {}
    __device__ __forceinline__ int start(int c) const { return c * each + c * more / n; }  // c, more < n <= 256
    __device__ __forceinline__ int owner(int f) const  // the CTA that takes page f < total
    {
        int c = min(static_cast<int>(static_cast<float>(f) * n / total), n - 1);  // at most one off
        while (start(c) > f) --c;
        while (start(c + 1) <= f) ++c;
        return c;
    }
};

// What parts of a unit are weighted against, M being their largest reference.  Without a score M is -inf: the parts are
// then zeros, or NaN where every score was NaN, and keep that under the weight 2^(-inf - 0) = 0.
__device__ __forceinline__ float base_of(float M) { return M == -INFINITY ? 0.f : M; }

// The factor on a unit's sum of weighted values, and its lse, for the sum of weights L: 0 and -inf without a token
// (L = 0), NaN where L is.
__device__ __forceinline__ float out_factor(float v_scale, float L) { return L != 0.f ? v_scale / L : 0.f; }
__device__ __forceinline__ float lse_of(float M, float L)
{
    return L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
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

// The launch's page list: Kmax places a unit (selections), or the pages of every batch entry's sequence, head after
// head.  Units count from the launch's first batch entry.
template <int T>
struct List {
    const int* first;  // every page: the first page of each batch entry, and the total
    const int* seq;    // ... and its tokens
    int per, Hkv, nb;  // selections: places a unit (0: every page)
    __device__ __forceinline__ int batch_of(int f) const  // the last entry that starts at or before page f
    {
        int a = 0, z = nb - 1;
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if (first[m] <= f) a = m;
            else z = m - 1;
        }
        return a;
    }
    __device__ __forceinline__ int count(int b) const { return (seq[b] + T - 1) / T; }
    __device__ __forceinline__ int unit_of(int f) const
    {
        if (per) return f / per;
        const int b = batch_of(f);
        return b * Hkv + (f - first[b]) / count(b);
    }
    __device__ __forceinline__ void range(int u, int& beg, int& end) const
    {
        if (per) {
            beg = u * per;
            end = beg + per;
        } else {
            const int b = u / Hkv, n = count(b);
            beg = first[b] + (u - b * Hkv) * n;
            end = beg + n;
        }
    }
};

template <int D, int T, bool DUP>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_kernel(const Kv4AttnParams p)
{
    using Page = Kv4Page<D, T>;
    constexpr int kDepth = ring_depth(D);
    constexpr int kPages = kStep / T;  // pages of a step
    constexpr int kSlot = step_bytes(D);
    static_assert(kSlot == kPages * Page::kBytes, "a slot holds whole pages");
    constexpr int kWords = D / 32;   // code words of a lane's K row
    constexpr int kTiles = D / 16;   // m-tiles of O^T
    constexpr int kMine = D / 8;     // output channels of a lane's row group
    constexpr int kVWords = D / 64;  // code words of a lane's V token
    constexpr int kPartRow = part_row(D);
    constexpr int kChain = DUP ? 16 : 8;  // most steps of a unit that the tensor core adds up in a row: 32 products
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.G;
    const int N = gridDim.x, rank = blockIdx.x;
    float* part = reinterpret_cast<float*>(smem + part_offset(D));
    int* first = reinterpret_cast<int*>(smem + list_offset(D, G));
    int* tokens = first + p.nb + 1;

    if (tid < kWarps * kDepth) {
        mbar_init(&sh.full[tid / kDepth][tid % kDepth], kPages);
        fence_barrier_init();
    }
    if (tid < 2 * kWarps) sh.unit[tid] = -1;
    __syncwarp();  // converged for the aligned barrier
    if (p.C > 1) cluster_arrive();  // passed before anything reaches another CTA
    // Every input may come from the preceding kernels.  Where the caller vouches for seq_len and the table, a launch
    // over every page sums the lengths and looks its first pages up while the preceding kernel drains, and waits for
    // it before it reads a query or a page or stores anything but error bits.  That saves 1.2 to 2.6 us behind an
    // append (one 128K sequence, both calls: 40.0 -> 37.9 us).  A launch with selections waits first: the pages come
    // from them, and its table rows are not fetched ahead.
    const bool early = p.early != 0 && p.sel_idx == nullptr;
    if (!early) pdl_wait_then_release();

    // ---- the page list and this CTA's piece of it ------------------------------------------------------------
    int total = 0;
    if (p.C > 0 || p.sel_idx != nullptr) {
        if (p.C == 0) total = p.nb * p.Hkv * p.Kmax;
        __syncthreads();  // the barriers exist
    } else {
        // a sequence a thread
        static_assert(kKv4MaxBatch <= kThreads, "one pass sums the batch's pages");
        int seq = 0;
        if (tid < p.nb) seq = clamped_seq(p, p.b0 + tid, rank == 0);
        const int pages = (seq + T - 1) / T * p.Hkv;
        int inc = pages;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(kFullMask, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int v = sh.scan[w];
            if (w < warp) before += v;
            total += v;
        }
        if (tid < p.nb) {
            first[tid] = before + inc - pages;
            tokens[tid] = seq;
        }
        if (tid == 0) first[p.nb] = total;
        __syncthreads();
    }
    // places a unit has in the list: Kmax, or, with a cluster a unit, Pmax; 0: its pages, summed above
    const List<T> list{first, tokens, p.sel_idx != nullptr ? p.Kmax : p.C > 0 ? p.Pmax : 0, p.Hkv, p.nb};
    // (integer divisions are a large part of what comes before the first copy: a cluster's CTA makes few)
    int lo, hi, wlo, whi, first_unit;  // the CTA's piece, this warp's places in it (every stride-th step) and first unit
    int stride = kWarps * kPages;
    int unit_seq = 0;  // every page, a cluster a unit: its tokens
    if (p.C > 0) {  // a unit's places (every page: those its sequence fills) dealt to its C CTAs
        const int c = p.C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
        first_unit = p.C > 1 ? static_cast<int>(cluster_id()) : rank;
        int n = p.Kmax;
        if (p.sel_idx == nullptr) {
            unit_seq = clamped_seq(p, p.b0 + first_unit / p.Hkv, c == 0 && first_unit % p.Hkv == 0);
            n = (unit_seq + T - 1) / T;
        }
        lo = first_unit * list.per + n * c / p.C;  // (n <= 32768, C <= 16)
        hi = whi = first_unit * list.per + n * (c + 1) / p.C;
        wlo = lo + kPages * warp;
    } else {  // a run of the CTA's piece, so that a warp meets few units
        lo = hi = wlo = whi = first_unit = 0;
        stride = kPages;
        if (total > 0) {
            const Pieces pieces(total, min(N, total));  // no piece is empty: the CTAs behind have none
            if (tid == 0) sh.total = total;
            if (rank < pieces.n) {
                lo = pieces.start(rank);
                hi = pieces.start(rank + 1);
                const int each = (hi - lo) / kWarps, more = (hi - lo) % kWarps;
                wlo = lo + each * warp + more * warp / kWarps;
                whi = lo + each * (warp + 1) + more * (warp + 1) / kWarps;
                if (wlo < whi) first_unit = list.unit_of(wlo);
            }
        }
    }

    const int gid = lane >> 2, tig = lane & 3;
    const int head = DUP ? (gid & 3) : gid;            // the query head of this lane's column
    const int col0 = DUP ? ((2 * tig) & 3) : 2 * tig;  // the heads of its accumulator columns: col0, col0 + 1
    const int ra = gid ^ ((gid >> 1) & 1);   // the tokens of this lane's K rows: ra and ra + 8
    const int t0 = (2 * tig) ^ (tig & 1), t1 = t0 ^ 1;  // ... and of its V pairs: (t0, t1) and (t0 + 8, t1 + 8)
    const float lo_lane = tig < 2 ? 0.f : -1.f;  // G <= 4: the lanes whose columns carry the lo parts
    uint4 qv[D / 32];
    auto load_queries = [&](int u) {
        const kvmm_bf16* qh = p.q + ((static_cast<size_t>(p.b0) * p.Hkv + u) * G + head) * D + tig * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            qv[i] = head < G ? reinterpret_cast<const uint4*>(qh)[i] : make_uint4(0u, 0u, 0u, 0u);
    };

    // ---- this warp's steps: round r is pages wlo + r * stride .. + kPages - 1 -------------------------------------
    constexpr int kBatch = 32 / kPages;  // rounds looked up at once, a page a lane
    uint8_t* ring = smem + static_cast<size_t>(warp) * kDepth * kSlot;
    const unsigned rounds = wlo < whi ? static_cast<unsigned>(whi - wlo + stride - 1) / static_cast<unsigned>(stride) : 0u;
    const uint64_t policy = l2_policy_evict_first();
    // A lane's page of the batch that starts with round rb: where it is held, and its word (unit * 64 + valid tokens;
    // without tokens there is nothing to copy).  Two dependent loads (the place in the selection, the table entry)
    // that a warp waits for once in kBatch steps, while the others go on (looking up a batch ahead took the same time
    // and more registers).
    const uint8_t* src = p.kv4_pool;
    int pmeta = 0;
    auto look_up = [&](int rb) {
        // (unsigned: a place behind the last may pass 2^31)
        const unsigned at = static_cast<unsigned>(wlo) + static_cast<unsigned>(rb + lane / kPages) * stride + lane % kPages;
        pmeta = 0x7fffffc0;  // behind the piece: after every unit
        if (at >= static_cast<unsigned>(whi)) return;
        const int f = static_cast<int>(at);
        int b, h, lp, u, seq;
        size_t unit;
        if (p.C > 0 && p.sel_idx == nullptr) {
            u = first_unit;
            b = u / p.Hkv;
            h = u - b * p.Hkv;
            lp = f - u * p.Pmax;
            seq = unit_seq;
            unit = (static_cast<size_t>(p.b0 + b) * p.L + p.layer) * p.Hkv + h;
            pmeta = u * 64;
        } else if (p.sel_idx != nullptr) {
            u = p.C > 0 ? first_unit : f / p.Kmax;
            const int i = f - u * p.Kmax;
            b = u / p.Hkv;
            h = u - b * p.Hkv;
            unit = (static_cast<size_t>(p.b0 + b) * p.L + p.layer) * p.Hkv + h;
            const int n = p.sel_cnt[unit];
            lp = p.sel_idx[unit * p.Kmax + i];
            seq = p.seq_len[p.b0 + b];
            if (i == 0 && (n < 0 || n > p.Kmax || seq < 0 || seq > p.Pmax * T)) report(p.err, KVMM_ERR_OUT_OF_RANGE);
            pmeta = u * 64;
            if (i >= n) return;
            seq = min(max(seq, 0), p.Pmax * T);
            if (lp < 0 || lp >= (seq + T - 1) / T) {
                report(p.err, KVMM_ERR_OUT_OF_RANGE);
                return;
            }
        } else {  // (the sum of the page counts has told of lengths out of range)
            b = list.batch_of(f);
            seq = tokens[b];
            const int n = list.count(b);
            h = (f - first[b]) / n;
            lp = f - first[b] - h * n;
            u = b * p.Hkv + h;
            unit = (static_cast<size_t>(p.b0 + b) * p.L + p.layer) * p.Hkv + h;
            pmeta = u * 64;
        }
        const int32_t phys = p.block_table[unit * p.Pmax + lp];
        if (phys < 0 || phys >= p.n_phys) {
            report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
            return;
        }
        src = p.kv4_pool + static_cast<size_t>(phys) * Page::kBytes;
        pmeta += min(T, seq - lp * T);
    };
    // this lane's copy of a step: the places its page and word go to, slot 0
    const unsigned my_round = static_cast<unsigned>(lane) / kPages, my_tile = static_cast<unsigned>(lane) % kPages;
    const uint32_t bar_at = smem_addr(&sh.full[warp][0]);
    const uint32_t meta_at = smem_addr(&sh.meta[warp][0]) + my_tile * 4;
    const uint32_t copy_at = smem_addr(ring) + my_tile * Page::kBytes;
    auto issue = [&](unsigned r) {  // start the copies of round r
        const unsigned k = r % kBatch;
        if (k == 0 && r != 0) look_up(static_cast<int>(r));
        if (k == my_round) {
            const uint32_t slot = r % kDepth;
            const int nv = pmeta & 63;
            if (kPages == 2) {
                sts_u32(meta_at + slot * 8, pmeta);
            } else {
                sts_u32(meta_at + slot * 8, pmeta - nv + min(nv, 16));
                sts_u32(meta_at + slot * 8 + 4, pmeta - nv + max(nv - 16, 0));
            }
            mbar_arrive_expect_tx_at(bar_at + slot * 8, nv > 0 ? Page::kBytes : 0);
            if (nv > 0) bulk_copy_g2s_hint_at(copy_at + slot * kSlot, src, Page::kBytes, bar_at + slot * 8, policy);
        }
    };
    if (!early && (p.C > 0 || wlo < whi)) load_queries(first_unit);  // on their way while the pages are looked up
    look_up(0);
    if (early) pdl_wait_then_release();
    if (p.C == 0 && p.sel_idx == nullptr) {
        // sequences without a token: their results are written here, spread over the CTAs
        for (int b = rank; b < p.nb; b += N) {
            if (tokens[b] != 0) continue;
            float* o = p.out + static_cast<size_t>(p.b0 + b) * p.Hq * D;
            for (int e = tid; e < p.Hq * D; e += kThreads) o[e] = 0.f;
            if (p.lse)
                for (int e = tid; e < p.Hq; e += kThreads) p.lse[static_cast<size_t>(p.b0 + b) * p.Hq + e] = -INFINITY;
        }
    }
    if (p.C == 0 && lo >= hi) return;  // (a cluster's CTA without a page takes part in its merge)
    if (early && (p.C > 0 || wlo < whi)) load_queries(first_unit);
#pragma unroll
    for (unsigned r = 0; r < kDepth; ++r)
        if (r < rounds) issue(r);

    // this lane's places in a page: its K row and scales, its V pairs' rows and scales
    const uint32_t ring_at = smem_addr(ring);
    const uint32_t k_off = ra * Page::kRow + tig * (D / 8), ks_off = ra * Page::kGroups + (D == 128 ? 2 * tig : tig);
    const uint32_t v0_off = t0 * Page::kRow + gid * (D / 16), v1_off = t1 * Page::kRow + gid * (D / 16);
    const uint32_t vs0_off = t0 * Page::kGroups + gid * kMine / 16, vs1_off = t1 * Page::kGroups + gid * kMine / 16;
    unsigned r = 0;

    auto part_at = [&](int k) {  // in bytes
        return k & 1 ? static_cast<unsigned>(k >> 1) * (kDepth * kSlot)
                     : static_cast<unsigned>(part_offset(D)) + static_cast<unsigned>(k >> 1) * (G * kPartRow * sizeof(float));
    };

    for (int u = first_unit; p.C > 0 || wlo < whi; ++u) {
        int ubeg, uend;
        list.range(u, ubeg, uend);
        if (uend == ubeg) continue;  // an empty sequence (a page of another follows: hi is beyond)
        // queries: halves of the lane's channels of its head, scaled by a power of two
        uint32_t qf[2 * kTiles];
        float zf0, zf1;
        {
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
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
                const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) qf[4 * i + k] = pack_half2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
            }
            // > 0: a masked score of -inf stays -inf under it
            zf0 = fmaxf(__shfl_sync(kFullMask, down, 4 * col0), FLT_MIN);
            zf1 = fmaxf(__shfl_sync(kFullMask, down, 4 * (col0 + 1)), FLT_MIN);
        }

        float o[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        // The tensor core rounds its sums toward zero: over a run of n products outputs come out too small by n * 2^-26 or
        // so (1.1e-6 at 63).  A longer run than kChain has its steps' sums added in fp32, rounded to nearest (32 ragged
        // sequences, 80 products: error against 64 bits 1.5e-6 -> 3.3e-7, 83.8 -> 85.8 us; every step of every run that
        // way: 13.4 -> 14.0 us for 64 pages of 32 and five heads).
        const bool long_run =
            (p.C > 0 ? static_cast<int>(rounds) * kPages : min(uend, whi) - max(ubeg, wlo)) > kChain * kPages;
        // One step.  FULL: both tiles are the unit's and have all their tokens (nearly every step: without its masks and
        // branches, every page of 32 sequences up to 16K tokens takes 87 us, with them 95).  APART: its
        // sums are added in fp32.
        auto step = [&](auto whole_step, auto apart, const uint32_t pg, const int nv0, const int nv1) {
            constexpr bool full = decltype(whole_step)::value;
            // tile j: tokens 16j .. 16j + 15 of the step, in page j (or the second half of the page)
            constexpr int kTile = kPages == 2 ? Page::kBytes : 16 * Page::kRow;
            constexpr int kTileScales = kPages == 2 ? Page::kBytes : 16 * Page::kGroups;
            const bool two = full || nv1 != 0;
            // ---- scores before their factor: x[j] = token ra of tile j with heads col0, col0 + 1, then token ra + 8
            float x[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j == 1 && !two) {
                    x[1][0] = x[1][1] = x[1][2] = x[1][3] = -INFINITY;
                    break;
                }
                float c[4] = {};
                uint32_t wa[kWords], wb[kWords], sa[kWords], sb[kWords];
                auto keys = [&](auto jc) {
                    constexpr int kAt = decltype(jc)::value * kTile, kSc = Page::kKeyScales + decltype(jc)::value * kTileScales;
                    if constexpr (D == 128) {
                        const uint4 y = lds_v4<kAt>(pg + k_off), z = lds_v4<kAt + 8 * Page::kRow>(pg + k_off);
                        wa[0] = y.x, wa[1] = y.y, wa[2] = y.z, wa[3] = y.w;
                        wb[0] = z.x, wb[1] = z.y, wb[2] = z.z, wb[3] = z.w;
                        // scale groups 2 tig and 2 tig + 1
                        const uint32_t ha = e4m3x2_to_half2(lds_u16<kSc>(pg + ks_off));
                        const uint32_t hb = e4m3x2_to_half2(lds_u16<kSc + 8 * Page::kGroups>(pg + ks_off));
                        sa[0] = sa[1] = prmt(ha, ha, 0x1010);
                        sa[2] = sa[3] = prmt(ha, ha, 0x3232);
                        sb[0] = sb[1] = prmt(hb, hb, 0x1010);
                        sb[2] = sb[3] = prmt(hb, hb, 0x3232);
                    } else {
                        const uint2 y = lds_v2<kAt>(pg + k_off), z = lds_v2<kAt + 8 * Page::kRow>(pg + k_off);
                        wa[0] = y.x, wa[1] = y.y, wb[0] = z.x, wb[1] = z.y;
                        const uint32_t hs = e4m3x2_to_half2(
                            prmt(lds_u8<kSc>(pg + ks_off), lds_u8<kSc + 8 * Page::kGroups>(pg + ks_off), 0x0040));
                        sa[0] = sa[1] = prmt(hs, hs, 0x1010);
                        sb[0] = sb[1] = prmt(hs, hs, 0x3232);
                    }
                };
                if (j == 0) keys(std::integral_constant<int, 0>{});
                else keys(std::integral_constant<int, 1>{});
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    mma_f16_16816(c, half2_mul(e2m1x2_to_half2<0>(wa[w]), sa[w]),
                                  half2_mul(e2m1x2_to_half2<0>(wb[w]), sb[w]),
                                  half2_mul(e2m1x2_to_half2<1>(wa[w]), sa[w]),
                                  half2_mul(e2m1x2_to_half2<1>(wb[w]), sb[w]), qf[4 * w], qf[4 * w + 1]);
                    mma_f16_16816(c, half2_mul(e2m1x2_to_half2<2>(wa[w]), sa[w]),
                                  half2_mul(e2m1x2_to_half2<2>(wb[w]), sb[w]),
                                  half2_mul(e2m1x2_to_half2<3>(wa[w]), sa[w]),
                                  half2_mul(e2m1x2_to_half2<3>(wb[w]), sb[w]), qf[4 * w + 2], qf[4 * w + 3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = c[i];
                if (!full) {  // selected, not multiplied: what the page holds there may be anything
                    if (ra >= (j == 0 ? nv0 : nv1)) x[j][0] = x[j][1] = -INFINITY;
                    if (ra + 8 >= (j == 0 ? nv0 : nv1)) x[j][2] = x[j][3] = -INFINITY;
                }
            }
            // ---- probabilities against a reference per head, raised only when a score exceeds it by more than
            // kSlack (one vote instead of a reduction a step).  The reference lies kLift below the maximum it
            // was taken from, so a probability is at most 2^(kSlack + kLift) = 2^15, and fp16 hi + lo holds it
            // to 2^-22 of itself or 2^-25 * 2^-kLift of the largest.
            constexpr float kSlack = 8.f, kLift = 7.f;
            float mx0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])) * zf0;
            float mx1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])) * zf1;
            if (!__all_sync(kFullMask, mx0 <= m0 + (kSlack + kLift) && mx1 <= m1 + (kSlack + kLift))) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, off));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, off));
                }
                // every step has a valid token, so the references are finite from the first one on
                const float n0 = fmaxf(m0, mx0 - kLift), n1 = fmaxf(m1, mx1 - kLift);
                const float a0 = fast_exp2(m0 - n0), a1 = fast_exp2(m1 - n1);
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
            uint32_t bh[2][2], bl[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p0 = fast_exp2(fmaf(x[j][0], zf0, -m0)), p1 = fast_exp2(fmaf(x[j][1], zf1, -m1));
                const float p2 = fast_exp2(fmaf(x[j][2], zf0, -m0)), p3 = fast_exp2(fmaf(x[j][3], zf1, -m1));
                l0 += p0 + p2;
                l1 += p1 + p3;
                const uint32_t h01 = pack_half2(p0, p1), h23 = pack_half2(p2, p3);
                if (DUP) {  // columns 0-3 carry hi, 4-7 lo: p less its hi part in the latter's lanes
                    bh[j][0] = movmatrix_trans(pack_half2(fmaf(half_lo(h01), lo_lane, p0), fmaf(half_hi(h01), lo_lane, p1)));
                    bh[j][1] = movmatrix_trans(pack_half2(fmaf(half_lo(h23), lo_lane, p2), fmaf(half_hi(h23), lo_lane, p3)));
                } else {
                    bh[j][0] = movmatrix_trans(h01);
                    bh[j][1] = movmatrix_trans(h23);
                    bl[j][0] = movmatrix_trans(pack_half2(p0 - half_lo(h01), p1 - half_hi(h01)));
                    bl[j][1] = movmatrix_trans(pack_half2(p2 - half_lo(h23), p3 - half_hi(h23)));
                }
            }
            // ---- values: channels gid * kMine .. + kMine - 1 of tokens t0, t1, t0 + 8, t1 + 8 of a tile -----------
            // byte b of an even / odd word: channel 2b / 2b + 1 of a token pair
            uint32_t ev01[2][kVWords], od01[2][kVWords], ev23[2][kVWords], od23[2][kVWords], s01[2], s23[2];
            auto load = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                constexpr int kAt = Page::kValues + j * kTile, kSc = Page::kValueScales + j * kTileScales;
                uint32_t w[4][kVWords], sc[4];
                if constexpr (D == 128) {
                    const uint2 y0 = lds_v2<kAt>(pg + v0_off), y1 = lds_v2<kAt>(pg + v1_off);
                    const uint2 y2 = lds_v2<kAt + 8 * Page::kRow>(pg + v0_off), y3 = lds_v2<kAt + 8 * Page::kRow>(pg + v1_off);
                    w[0][0] = y0.x, w[0][1] = y0.y, w[1][0] = y1.x, w[1][1] = y1.y;
                    w[2][0] = y2.x, w[2][1] = y2.y, w[3][0] = y3.x, w[3][1] = y3.y;
                } else {
                    w[0][0] = lds_u32<kAt>(pg + v0_off), w[1][0] = lds_u32<kAt>(pg + v1_off);
                    w[2][0] = lds_u32<kAt + 8 * Page::kRow>(pg + v0_off), w[3][0] = lds_u32<kAt + 8 * Page::kRow>(pg + v1_off);
                }
                sc[0] = lds_u8<kSc>(pg + vs0_off), sc[1] = lds_u8<kSc>(pg + vs1_off);
                sc[2] = lds_u8<kSc + 8 * Page::kGroups>(pg + vs0_off), sc[3] = lds_u8<kSc + 8 * Page::kGroups>(pg + vs1_off);
                if (!full) {  // a scale of zero: codes are always finite
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (((k & 1) ? t1 : t0) + (k >> 1) * 8 >= (j == 0 ? nv0 : nv1)) sc[k] = 0u;
                }
                s01[j] = e4m3x2_to_half2(prmt(sc[0], sc[1], 0x0040));
                s23[j] = e4m3x2_to_half2(prmt(sc[2], sc[3], 0x0040));
#pragma unroll
                for (int i = 0; i < kVWords; ++i) {
                    ev01[j][i] = (w[0][i] & 0x0f0f0f0fu) | ((w[1][i] << 4) & 0xf0f0f0f0u);
                    od01[j][i] = ((w[0][i] >> 4) & 0x0f0f0f0fu) | (w[1][i] & 0xf0f0f0f0u);
                    ev23[j][i] = (w[2][i] & 0x0f0f0f0fu) | ((w[3][i] << 4) & 0xf0f0f0f0u);
                    od23[j][i] = ((w[2][i] >> 4) & 0x0f0f0f0fu) | (w[3][i] & 0xf0f0f0f0u);
                }
            };
            // m-tile i of token tile j: rows gid are channel i of the lane's, rows gid + 8 channel kTiles + i
            auto product = [&](auto ic, const int j, float (&c)[4]) {
                constexpr int a = decltype(ic)::value, b = kTiles + a;  // channels
                constexpr int ba = (a % 8) / 2, bb = (b % 8) / 2;
                const uint32_t xa = (a & 1) ? od01[j][a / 8] : ev01[j][a / 8], xb = (b & 1) ? od01[j][b / 8] : ev01[j][b / 8];
                const uint32_t ya = (a & 1) ? od23[j][a / 8] : ev23[j][a / 8], yb = (b & 1) ? od23[j][b / 8] : ev23[j][b / 8];
                const uint32_t a0 = half2_mul(e2m1x2_to_half2<ba>(xa), s01[j]), a1 = half2_mul(e2m1x2_to_half2<bb>(xb), s01[j]);
                const uint32_t a2 = half2_mul(e2m1x2_to_half2<ba>(ya), s23[j]), a3 = half2_mul(e2m1x2_to_half2<bb>(yb), s23[j]);
                mma_f16_16816(c, a0, a1, a2, a3, bh[j][0], bh[j][1]);
                if (!DUP) mma_f16_16816(c, a0, a1, a2, a3, bl[j][0], bl[j][1]);
            };
            auto each = [&](auto f) {
                f(std::integral_constant<int, 0>{});
                f(std::integral_constant<int, 1>{});
                f(std::integral_constant<int, 2>{});
                f(std::integral_constant<int, 3>{});
                if constexpr (kTiles == 8) {
                    f(std::integral_constant<int, 4>{});
                    f(std::integral_constant<int, 5>{});
                    f(std::integral_constant<int, 6>{});
                    f(std::integral_constant<int, 7>{});
                }
            };
            load(std::integral_constant<int, 0>{});
            if constexpr (decltype(apart)::value) {
                load(std::integral_constant<int, 1>{});
                each([&](auto ic) {
                    float c[4] = {};
                    product(ic, 0, c);
                    product(ic, 1, c);
                    add4(o[decltype(ic)::value], c);
                });
            } else {
                each([&](auto ic) { product(ic, 0, o[decltype(ic)::value]); });
                if (two) {
                    load(std::integral_constant<int, 1>{});
                    each([&](auto ic) { product(ic, 1, o[decltype(ic)::value]); });
                }
            }
        };
        while (r < rounds) {
            const uint32_t slot = r % kDepth;
            if (__any_sync(kFullMask, !mbar_wait_bounded(&sh.full[warp][slot], (r / kDepth) & 1, kWaitNs))) {
                if (lane == 0) report(p.err, KVMM_ERR_TIMEOUT);  // the remaining pages are dropped
                for (unsigned k = r; k < min(rounds, r + kDepth); ++k)  // what is in flight lands before the CTA leaves
                    mbar_wait_bounded(&sh.full[warp][k % kDepth], (k / kDepth) & 1, 100000000ull);
                __syncwarp();
                r = rounds;
                break;
            }
            const int2 meta = sh.meta[warp][slot];
            const uint32_t pg = ring_at + slot * kSlot;
            if (meta.x == u * 64 + 16 && meta.y == u * 64 + 16) {
                if (long_run) step(std::true_type{}, std::true_type{}, pg, 16, 16);
                else step(std::true_type{}, std::false_type{}, pg, 16, 16);
            } else {
                if ((meta.x >> 6) > u) break;  // the step is of a later unit
                const int nv0 = (meta.x >> 6) == u ? meta.x & 63 : 0, nv1 = (meta.y >> 6) == u ? meta.y & 63 : 0;
                if (nv0 > 0) step(std::false_type{}, std::false_type{}, pg, nv0, nv1);
                // the first page is of the unit before, or could not be read
                else if (kPages == 2 && nv1 > 0) step(std::false_type{}, std::false_type{}, pg + Page::kBytes, nv1, 0);
                if ((meta.y >> 6) > u && (meta.y & 63) != 0) break;  // the second page is of a later unit
            }
            ++r;
            __syncwarp();
            if (r + kDepth - 1 < rounds) {
                fence_proxy_async_shared();  // this slot's reads before the copy that refills it
                issue(r + kDepth - 1);
            }
        }

        const bool last = p.C > 0 || uend >= whi;
        if (!last) {  // the next unit's queries are on their way while this one's results are stored
            int nu = u + 1, b0, b1;
            for (list.range(nu, b0, b1); b0 == b1; list.range(nu, b0, b1)) ++nu;  // (a unit with pages follows: whi is beyond)
            load_queries(nu);
        }
        // ---- the unit ends here (or this warp's piece of it) ------------------------------------------------------
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(kFullMask, l0, off);
            l1 += __shfl_xor_sync(kFullMask, l1, off);
        }
        // a unit that this warp has alone is written out, else its part is stored
        const bool whole = p.C == 0 && ubeg >= wlo && uend <= whi;
        const int k = 2 * warp + (last ? 1 : 0);
        const size_t row = (static_cast<size_t>(p.b0) * p.Hkv + u) * G;
        __syncwarp();  // the last reads of the ring
        auto results = [&](auto put) {  // put(which of the lane's heads, channel of its row group, value)
#pragma unroll
            for (int i = 0; i < (DUP ? kTiles / 2 : kTiles); ++i) {
                float v[4];
                int d = i;
                if (DUP) {  // hi + lo: the lanes with the hi columns take the first half of the tiles, the others the rest
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float give = tig < 2 ? o[i + kTiles / 2][j] : o[i][j];
                        const float keep = tig < 2 ? o[i][j] : o[i + kTiles / 2][j];
                        v[j] = keep + __shfl_xor_sync(kFullMask, give, 2);
                    }
                    if (tig >= 2) d += kTiles / 2;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = o[i][j];
                }
                if (col0 < G) {
                    put(0, d, v[0]);
                    put(0, d + kTiles, v[2]);
                }
                if (col0 + 1 < G) {
                    put(1, d, v[1]);
                    put(1, d + kTiles, v[3]);
                }
            }
        };
        const bool tell = gid == 0 && (!DUP || tig < 2);
        if (whole) {
            float* dst = p.out + (row + col0) * D + gid * kMine;
            const float f[2] = {out_factor(p.v_scale, l0), out_factor(p.v_scale, l1)};
            results([&](int h, int d, float v) { dst[h * D + d] = v * f[h]; });
            if (p.lse && tell) {
                if (col0 < G) p.lse[row + col0] = lse_of(m0, l0);
                if (col0 + 1 < G) p.lse[row + col0 + 1] = lse_of(m1, l1);
            }
        } else {  // (zeros where the warp had no page of the unit)
            const uint32_t dst = smem_addr(smem) + part_at(k) + (col0 * kPartRow + gid * (kMine + 1)) * sizeof(float);
            results([&](int h, int d, float v) { sts_u32(dst + (h * kPartRow + d) * sizeof(float), __float_as_uint(v)); });
            if (lane == 0) sh.unit[k] = u;
            if (tell) {
                sh.m[k][col0] = m0;
                sh.m[k][col0 + 1] = m1;
                sh.l[k][col0] = l0;
                sh.l[k][col0 + 1] = l1;
            }
        }
        if (last) break;
    }
    __syncthreads();  // the parts are stored

    if (p.C > 0) {
        const uint32_t ring0 = smem_addr(smem);
        const size_t row = (static_cast<size_t>(p.b0) * p.Hkv + first_unit) * G;
        auto write = [&](int e, float O, float M, float L) {
            p.out[row * D + e] = O * out_factor(p.v_scale, L);
            if (p.lse && e % D == 0) p.lse[row + e / D] = lse_of(M, L);
        };
        // one output channel over the warps' parts: unnormalised, with the reference and the sum
        auto combine = [&](int e, float& M, float& L) {
            const int g = e / D, d = e % D;
            const uint32_t at = ring0 + (g * kPartRow + d / kMine * (kMine + 1) + d % kMine) * sizeof(float);
            float m[kWarps];
            M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                m[w] = sh.m[2 * w + 1][g];
                M = fmaxf(M, m[w]);
            }
            const float base = base_of(M);
            L = 0.f;
            float O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = fast_exp2(m[w] - base);
                const float y = __uint_as_float(lds_u32<0>(at + w * (kDepth * kSlot)));
                L = fmaf(sh.l[2 * w + 1][g], f, L);
                O = fmaf(y, f, O);
            }
            return O;
        };
        if (p.C == 1) {
            for (int e = tid; e < G * D; e += kThreads) {
                float M, L;
                const float O = combine(e, M, L);
                write(e, O, M, L);
            }
            return;
        }
        // the unit's CTAs are a cluster: each stores, into every other, its references and sums and the slice of
        // its outputs that the other owns; after one cluster barrier every CTA combines its slice
        const int C = p.C, rc = static_cast<int>(cluster_ctarank());
        const int slice = (G * D + C - 1) / C;
        cluster_wait();
        for (int e = tid; e < G * D; e += kThreads) {
            const int c = e / slice;
            float M, L;
            const float O = combine(e, M, L);
            st_dsmem_f32(&sh.recv[rc * slice + (e - c * slice)], c, O);
            if (e % D == 0)
                for (int k = 0; k < C; ++k) {
                    st_dsmem_f32(&sh.rstat[rc][e / D], k, M);
                    st_dsmem_f32(&sh.rstat[rc][8 + e / D], k, L);
                }
        }
        __syncwarp();
        cluster_sync();
        for (int i = tid; i < slice; i += kThreads) {
            const int e = rc * slice + i, g = e / D;
            if (e >= G * D) break;
            float M = -INFINITY, L = 0.f, O = 0.f;
            for (int c = 0; c < C; ++c) M = fmaxf(M, sh.rstat[c][g]);
            const float base = base_of(M);
            for (int c = 0; c < C; ++c) {
                const float f = exp2f(sh.rstat[c][g] - base);
                L = fmaf(sh.rstat[c][8 + g], f, L);
                O = fmaf(sh.recv[c * slice + i], f, O);
            }
            write(e, O, M, L);
        }
        return;
    }

    // ---- units that fell on several warps: the parts of one follow one another ----------------------------------
    const int mine = sh.unit[lane];  // a part a lane
    const unsigned there = __ballot_sync(kFullMask, mine >= 0);
    const unsigned behind = lane == 31 ? 0u : there & (~0u << (lane + 1));
    const int next = __shfl_sync(kFullMask, mine, behind ? __ffs(behind) - 1 : lane);
    const bool ends = mine >= 0 && (behind == 0u || next != mine);  // the last part of its unit
    bool whole = false, begins = true;                              // the unit lies in this CTA; begins in it
    if (mine >= 0) {
        int ubeg, uend;
        list.range(mine, ubeg, uend);
        whole = ubeg >= lo && uend <= hi;
        begins = ubeg >= lo;
    }
    const int rank_of = __popc(there & ((1u << lane) - 1u));
    if (warp == 0 && mine >= 0) sh.at[rank_of] = static_cast<int>(part_at(lane));
    const unsigned ending = __ballot_sync(kFullMask, ends);
    // the CTA's two places in the workspace: for the unit that began before, and the one that goes on
    float* const slot0 = p.partial + static_cast<size_t>(rank) * 2 * kv4_partial_floats(D);
    if (warp < G) {  // a head a warp: the parts' weights
        float m = -INFINITY, l = 0.f;
        if (mine >= 0) m = sh.m[lane][warp], l = sh.l[lane][warp];
        const unsigned done = ending & ((1u << lane) - 1u), open = ending & (~0u << lane);
        const int s = done ? 32 - __clz(done) : 0, t = open ? __ffs(open) - 1 : 31;  // the lanes of this part's unit
        float M = m;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float x = __shfl_up_sync(kFullMask, M, off);
            if (lane - off >= s) M = fmaxf(M, x);
        }
        M = __shfl_sync(kFullMask, M, t);
        const float f = exp2f(m - base_of(M));
        float L = l * f;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float x = __shfl_up_sync(kFullMask, L, off);
            if (lane - off >= s) L += x;
        }
        L = __shfl_sync(kFullMask, L, t);
        if (mine >= 0) sh.weight[rank_of][warp] = whole ? f * out_factor(p.v_scale, L) : f;
        if (ends) {
            if (whole) {
                if (p.lse)
                    p.lse[(static_cast<size_t>(p.b0) * p.Hkv + mine) * G + warp] = lse_of(M, L);
            } else {
                float* stat = slot0 + (begins ? kv4_partial_floats(D) : 0) + 8 * D + warp;
                stat[0] = M;
                stat[8] = L;
            }
        }
    }
    const unsigned whole_mask = __ballot_sync(kFullMask, whole), begin_mask = __ballot_sync(kFullMask, begins);
    __syncthreads();
    for (int e = tid; e < G * D; e += kThreads) {
        const int g = e / D, d = e % D;
        const uint32_t here = smem_addr(smem) + (g * kPartRow + d / kMine * (kMine + 1) + d % kMine) * sizeof(float);
        int i = 0;
#pragma unroll 1
        for (unsigned left = ending; left != 0u; left &= left - 1u) {  // a unit a round
            const int t = __ffs(left) - 1, to = __popc(there & ((2u << t) - 1u));
            float* dst = whole_mask >> t & 1u ? p.out + (static_cast<size_t>(p.b0) * p.Hkv + sh.unit[t]) * G * D
                                              : slot0 + (begin_mask >> t & 1u ? kv4_partial_floats(D) : 0);
            float acc = 0.f;
#pragma unroll 4
            for (; i < to; ++i) acc = fmaf(sh.weight[i][g], __uint_as_float(lds_u32<0>(here + sh.at[i])), acc);
            dst[e] = acc;
        }
    }
    // units that several CTAs share: the first of them, and how many
    int shared_unit[2], c0 = 0, np = 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const unsigned those = there & ~whole_mask & (side ? begin_mask : ~begin_mask);
        shared_unit[side] = those ? sh.unit[__ffs(those) - 1] : -1;
    }
    if (tid < 2) {
        sh.span[tid][1] = 0;
        const int u = tid ? shared_unit[1] : shared_unit[0];
        if (u >= 0) {
            int beg, end;
            list.range(u, beg, end);
            const Pieces pieces(sh.total, min(N, sh.total));
            c0 = pieces.owner(beg);
            np = pieces.owner(end - 1) - c0 + 1;
        }
    }
    __syncthreads();  // this CTA's parts are stored

    // ---- units that fell on several CTAs: whoever stored the last part combines them ---------------------------
    // A unit's counter is that of the first CTA it lies in, which can be the first for one such unit only.
    if (np > 0) {  // (threads 0 and 1)
        // release: this CTA's parts, stored before the barrier above; acquire: the other CTAs'
        int before;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.counter + c0) : "memory");
        if (before == np - 1) {
            p.counter[c0] = 0;  // as the next call has to find it
            sh.span[tid][0] = c0;
            sh.span[tid][1] = np;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int c0 = sh.span[side][0], np = sh.span[side][1];
        if (np == 0) continue;
        const size_t row = (static_cast<size_t>(p.b0) * p.Hkv + (side ? shared_unit[1] : shared_unit[0])) * G;
        // The first part is its CTA's last unit, the others are their CTAs' first.
        constexpr size_t kPart = kv4_partial_floats(D);
        const float* parts = p.partial + static_cast<size_t>(c0) * 2 * kPart;
        auto part_of = [&](int k) { return parts + (k == 0 ? kPart : static_cast<size_t>(2 * k) * kPart); };
        float* weight = reinterpret_cast<float*>(smem);  // [np][8], then the sums: where the rings were
        float* sum = weight + kKv4MaxCtas * 8;
        for (int i = tid; i < np * 8; i += kThreads) {
            const float* stat = part_of(i >> 3) + 8 * D + (i & 7);
            weight[i] = __ldcg(stat);
            sum[i] = __ldcg(stat + 8);
        }
        // a thread takes four channels of one head from every ngrp-th part, eight loads in flight
        const int nf4 = G * D / 4, ngrp = min(min(kThreads / nf4, kWarps), np);
        const int grp = tid / nf4, e = tid - grp * nf4, g = 4 * e / D;
        float4 x[8];
        auto load = [&](int k0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = k0 + i * ngrp;
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (grp < ngrp && k < np) x[i] = __ldcg(reinterpret_cast<const float4*>(part_of(k)) + e);
            }
        };
        load(grp);
        __syncthreads();
        if (warp < G) {
            float M = -INFINITY, L = 0.f;
            for (int k = lane; k < np; k += 32) M = fmaxf(M, weight[8 * k + warp]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, off));
            for (int k = lane; k < np; k += 32) {
                const float f = exp2f(weight[8 * k + warp] - base_of(M));
                weight[8 * k + warp] = f;
                L = fmaf(sum[8 * k + warp], f, L);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(kFullMask, L, off);
            if (lane == 0) {
                sh.l[0][warp] = out_factor(p.v_scale, L);
                if (p.lse) p.lse[row + warp] = lse_of(M, L);
            }
        }
        __syncthreads();
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = grp; k0 < np; k0 += 8 * ngrp) {
            if (k0 != grp) load(k0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = k0 + i * ngrp < np ? weight[8 * (k0 + i * ngrp) + g] : 0.f;
                a.x = fmaf(x[i].x, f, a.x);
                a.y = fmaf(x[i].y, f, a.y);
                a.z = fmaf(x[i].z, f, a.z);
                a.w = fmaf(x[i].w, f, a.w);
            }
        }
        if (grp < ngrp) reinterpret_cast<float4*>(part)[tid] = a;  // (ngrp <= kWarps: they fit where the parts were)
        __syncthreads();
        for (int i = tid; i < G * D; i += kThreads) {
            float O = 0.f;
            for (int k = 0; k < ngrp; ++k) O += part[k * G * D + i];
            p.out[row * D + i] = O * sh.l[0][i / D];
        }
        __syncthreads();
    }
}

// clusters of c CTAs of this kernel that the device holds at once
int clusters_at_once(void (*kernel)(Kv4AttnParams), size_t smem, int c)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c, 1, 1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

template <int D, int T>
cudaError_t launch(Kv4AttnParams p, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool dup = p.G <= 4;
    void (*kernel)(Kv4AttnParams) = dup ? kv4_attn_kernel<D, T, true> : kv4_attn_kernel<D, T, false>;
    // per thread and device: what the launches need to know of it
    struct Device {
        int dev = -1, sms = 0;
        bool ready[2] = {};  // by kernel
        int held[9][kKv4MaxCluster + 1] = {};  // clusters of c CTAs held at once, by group size; 0: not asked yet
    };
    static thread_local Device known;
    if (known.dev != dev) {
        known = Device{};
        e = cudaDeviceGetAttribute(&known.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known.dev = dev;
    }
    if (!known.ready[dup]) {  // the most any launch of this kernel takes, so that clusters can be asked for first
        const size_t most = smem_bytes(D, dup ? 4 : 8, kKv4MaxBatch);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        known.ready[dup] = true;
    }
    // batch entries of one launch: their page counts are summed in shared memory, and the list's length is an int
    const long long each = static_cast<long long>(p.Hkv) * (p.sel_idx ? p.Kmax : p.Pmax);  // <= 2^31
    long long room = (1ll << 30) / each;
    if (room > (1 << 24) / p.Hkv) room = (1 << 24) / p.Hkv;  // a unit's number and a count of tokens share a word
    const int step = room < 1 ? 1 : room < kKv4MaxBatch ? static_cast<int>(room) : kKv4MaxBatch;
    for (p.b0 = 0; p.b0 < p.B; p.b0 += step) {
        p.nb = p.B - p.b0 < step ? p.B - p.b0 : step;
        const long long units = static_cast<long long>(p.nb) * p.Hkv;
        // A cluster a unit, as many CTAs as all run at once and have 16 pages each, where the units are no more than
        // the SMs: with selections, or when a CTA's share of the longest sequence is short (kShortTiles).  What an
        // uneven batch then loses to its longest sequence is less than what dealing its pages evenly costs: the sum of
        // the lengths, the units that end inside a CTA and the merge through memory.  Six sequences of up to 1,914
        // tokens, 8 KV heads: 9.6 us against 16.0; at the border, sixteen of up to 4,096 19.2 against 24.7, four
        // of up to 16K 20.3 against 21.7, one of 64K 25.5 against 23.4.  Beyond it the SMs that whole clusters leave
        // empty (24 of 152) cost more: two of 60,000 tokens 40.8 against 33.6, one of 128K 44.1 against 35.0.
        const int places = p.sel_idx ? p.Kmax : p.Pmax;
        p.C = 0;
        if (units <= known.sms) {
            const size_t bare = smem_bytes(D, p.G, 0);
            int most = (places + kWarps - 1) / kWarps;
            if (most > kKv4MaxCluster) most = kKv4MaxCluster;
            p.C = 1;
            for (int c = 2; c <= most && units * c <= known.sms; ++c) {
                int& held = known.held[p.G][c];
                if (held == 0) {
                    held = clusters_at_once(kernel, bare, c);
                    if (held == 0) held = -1;
                }
                if (held >= units) p.C = c;
            }
            if (p.sel_idx == nullptr && (places + p.C - 1) / p.C * (T / 16) > kShortTiles) p.C = 0;
        }
        const size_t smem = smem_bytes(D, p.G, p.C == 0 && !p.sel_idx ? p.nb : 0);
        long long n = units * p.C;
        if (p.C == 0) {  // one CTA an SM, fewer when not every warp would get a page
            n = (each * p.nb + kWarps - 1) / kWarps;
            if (n > known.sms) n = known.sms;
            if (n > kKv4MaxCtas) n = kKv4MaxCtas;
        }
        if (p.C > 1)
            e = launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(n)), dim3(kThreads), smem, stream,
                                   static_cast<unsigned>(p.C), p);
        else
            e = launch_pdl(kernel, dim3(static_cast<unsigned>(n)), dim3(kThreads), smem, stream, p);
        if (e != cudaSuccess) return e;
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
