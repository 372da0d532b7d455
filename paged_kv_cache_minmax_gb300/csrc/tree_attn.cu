// tree_attn.cu -- attention of a tree of drafted tokens over the paged cache.
//
// The query rows of one (batch, KV head), nodes x heads of the group, are the
// M axis of the tensor cores: tiles of 128 rows against blocks of 128 tokens,
//     S = Q K^T      [128 x 128], fp32 in tensor memory
//     P = exp2(S - m), as two bf16 halves, written over S in tensor memory
//     O += P V       [128 x D], fp32 in tensor memory, a product for each half
// with m a running reference of each row: it moves, and O and the sum are
// rescaled, only when a score passes it by 2^8, so weights stay below 2^8.
//
// A weight keeps 16 bits, as in the decode attention: one rounded to a single bf16
// adds 1.1e-3 to the 1.7e-3 that the output's own rounding is off (against 64 bits,
// relative), two halves nothing that shows.  The second half is a second product:
// one 128K sequence, 64 nodes x 4 heads 147 us instead of 118 (calls in a row), 16
// ragged ones of up to 16K 133 instead of 130, 128 selected pages 25.3 instead of
// 23.0, one of 4K 13.6 instead of 12.4.
//
// The pages are in the form the tensor cores take: a key page [T][D] is T
// K-major rows of Q K^T's second operand, a value page [D][T] D K-major rows
// of P V's, each 16 tokens wide or twice that.  TMA copies them with the
// swizzle of their rows (128 bytes for keys, 32 or 64 for values).
//
// A CTA's warps: two groups of four for the softmax of two streams (a thread a
// row), one that copies, one whose elected thread issues the products.  The
// streams alternate on the tensor cores: two row tiles over the same blocks, or,
// with at most 128 rows, one tile over every other block, joined at the end from
// tensor memory.  128 rows are the tensor cores' own tile; fewer rows leave part
// of it unused, which costs nothing as long as the memory is the bound: a block
// (64 KB with 128 channels) takes 2,800 cycles at a copy's rate, its products
// about 2,300 a tile (Q K^T 650, each half's P V 850), its softmax some 2,000 (128
// exponentials a row at 16 a clock and SM).  Two tiles take 4,500 of products, so the
// largest trees are bound by them.
//
// Short units take a cluster of CTAs each, joined through distributed shared
// memory.  Otherwise the blocks of all units are dealt evenly to one CTA an SM,
// whatever the sequences' lengths; a unit that falls on several CTAs leaves parts
// in the workspace, which a second launch joins.
//
// Times (us of a launch in a graph; the floor is the bytes at a copy's rate): one 128K
// sequence, 8 KV heads, 64 nodes x 4 heads 137 (79; 137 GFLOP, 1,000 TFLOP/s); 16
// ragged sequences of up to 16K tokens, pages of 32, 13 nodes x 5 heads 135 (116);
// eight sequences, 128 selected pages, 16 nodes 24.6 (10.3); one of 4K 13.3 (2.5), which
// is latency: lengths, table entry, first block 3.7, products and softmax 5, join 3.
#include <cstdint>

#include "kernels.h"
#include "tcgen05.cuh"

namespace kvmm {
namespace {

constexpr int kThreads = 384;    // 8 softmax warps, the copying warp, the issuing warp, two that only share registers
constexpr int kTokens = 128;     // tokens of a block
constexpr int kRing = 8;         // blocks whose masks are held (see copy_pages)
constexpr int kNoNode = 1 << 20; // an entry that holds no node
constexpr int kUnitsAtOnce = 2048;
constexpr int kShort = 128;      // blocks x tiles of a unit up to which a cluster takes it
// Steps of a stream whose products tensor memory sums.  Its additions round toward zero, 16 a step: over 64 steps of sums that
// grow steadily the result is low by up to 2^-14 (half of 1,024 x 2^-23).  Then the sums go to the workspace, where they are
// added to the nearest.  (Without: 2^20 tokens of positive values in one CTA 2.1e-3 low, more than half of what rounding to
// bf16 may do.)
constexpr int kRun = kShort / 2;

struct Launch {
    TreeAttnParams p;
    int b0, nb;      // batch entries of this launch
    int tiles;       // row tiles of a unit: 1 or 2
    int groups;      // units of one (batch, KV head): 1 or 2
    int units;       // nb * Hkv * groups
    int tile_rows;   // rows of a tile in the workspace
    int cluster;     // CTAs of a unit, one cluster; 0: the blocks of all units are dealt evenly to the CTAs
    int by_unit;     // (dealt evenly) cut has an entry for each unit, else for each CTA
    int4* cut;       // a unit whose blocks fall on several CTAs (x -1: none): unit, first CTA, last CTA, rows
    float2* ml;      // [2 * CTAs][tiles][tile_rows] reference and sum
    float4* o;       // [2 * CTAs][tiles][D / 4][tile_rows]
    float4* run;     // [CTAs][2 streams][D / 4][tile_rows] sums of a stream's steps before the last kRun
};

struct Unit {
    int b, h;
    int seq, held;         // settled tokens, nodes with a place
    int row0, rows;        // rows of the unit among the nodes' rows
    int listed, entries;   // pages of settled tokens, all pages
    int blocks;
    size_t index;          // of the (batch, layer, KV head)
};

template <int T>
__device__ __forceinline__ Unit unit_of(const Launch& a, int w, bool tell)
{
    const TreeAttnParams& p = a.p;
    Unit u;
    const int g = w & (a.groups - 1), bh = w >> (a.groups - 1);  // (one or two groups)
    u.b = bh / p.Hkv;
    u.h = bh - u.b * p.Hkv;
    u.b += a.b0;
    u.index = (static_cast<size_t>(u.b) * p.L + p.layer) * p.Hkv + u.h;
    const int cap = p.Pmax * T;
    int n = p.n_nodes != nullptr ? p.n_nodes[u.b] : p.n_max;
    int cnt = p.sel_idx != nullptr ? p.sel_cnt[u.index] : 0;
    u.seq = p.seq_len[u.b];
    bool bad = u.seq < 0 || u.seq > cap || n < 0 || n > p.n_max || cnt < 0 || cnt > p.Kmax;
    u.seq = min(max(u.seq, 0), cap);
    n = min(max(n, 0), p.n_max);
    cnt = min(max(cnt, 0), p.Kmax);
    u.held = min(n, cap - u.seq);
    bad |= u.held < n;
    if (tell && bad) report(p.err, KVMM_ERR_OUT_OF_RANGE);
    u.row0 = g * a.tiles * 128;
    u.rows = min(max(n * p.G - u.row0, 0), a.tiles * 128);
    if (p.sel_idx != nullptr) {
        u.listed = cnt;
        u.entries = cnt + (u.held > 0 ? (u.seq + u.held - 1) / T - u.seq / T + 1 : 0);
    } else {
        u.listed = u.entries = (u.seq + u.held + T - 1) / T;
    }
    u.blocks = u.rows > 0 ? (u.entries * T + kTokens - 1) / kTokens : 0;
    return u;
}

// what a block shows: for each of its pages the slots of settled tokens, and the node in its first slot
struct BlockMask {
    uint32_t settled[kTokens / 16];
    int32_t node0[kTokens / 16];
    int32_t whole;  // every slot is a settled token's
    int32_t held;   // nodes of the sequence
    int32_t pages;  // up to the last that was copied (1 at least): what lies behind is not multiplied
};

struct Control {
    uint64_t full[10], empty[10], s_full[2], p_ready[2], q_ready[2], o_done[2], meet, drain;
    unsigned long long spoilt[2];  // nodes that have a value that is not finite, by the piece's parity
    uint32_t tmem;
    int32_t gave_up;
    int32_t w0, off0, left;
    int4 cut;
    Unit unit;  // w0
    int32_t sums[kThreads / 32];
    BlockMask mask[kRing];
    float2 ml[2][128];
};

template <int D>
struct Smem {
    static constexpr int kTile = 128 * D * 2;  // a tile of queries, a block of keys or of values
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kControl = (2 + kStages) * kTile;
    static constexpr size_t kBytes = kControl + sizeof(Control);
};
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "shared memory of a CTA");

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// wait for the phase; false once any warp of the CTA has given up
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int32_t* gave_up)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t spin = 0;; ++spin) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((spin & 63u) != 63u) continue;
        if (*gave_up != 0) return false;
        if (global_timer_ns() - t0 > 1000000000ull) {
            *gave_up = 1;
            return false;
        }
    }
}

// the CTA's run of blocks, piece by piece (a piece: blocks of one unit)
struct Walk {
    int w, off, left;   // unit, its next block, blocks of the run to come
    const Unit* first;  // unit w, as long as it is the run's first
};
template <int T>
__device__ __forceinline__ bool next_piece(const Launch& a, Walk& k, Unit& u, int& begin, int& count)
{
    if (k.left <= 0) return false;
    for (;; ++k.w, k.off = 0) {
        if (k.w >= a.units) return false;
        u = k.first != nullptr ? *k.first : unit_of<T>(a, k.w, false);
        k.first = nullptr;
        if (u.blocks > k.off) break;
    }
    begin = k.off;
    count = min(u.blocks - k.off, k.left);
    k.off += count;
    k.left -= count;
    return true;
}

// ---- the copying warp -------------------------------------------------------------
template <int D, int T>
__device__ void copy_pages(const Launch& a, const CUtensorMap* kmap, const CUtensorMap* vmap, uint8_t* smem, Control& c, Walk k)
{
    using S = Smem<D>;
    constexpr int kPages = kTokens / T;        // pages of a block
    constexpr int kBlocks = 32 / kPages;       // blocks whose pages the lanes look up at once
    constexpr uint32_t kPageBytes = T * D * 2;
    const int lane = threadIdx.x & 31, mine = lane % kPages;
    const TreeAttnParams& p = a.p;
    uint8_t* ring = smem + 2 * S::kTile;
    const uint64_t policy = l2_policy_evict_first();
    uint32_t item = 0, nth = 0;
    bool fine = true;
    Unit u;
    int begin, count;
    while (fine && next_piece<T>(a, k, u, begin, count)) {
        const int32_t* table = p.block_table + u.index * p.Pmax;
        const int32_t* sel = p.sel_idx != nullptr ? p.sel_idx + u.index * p.Kmax : nullptr;
        const int pages = (u.seq + T - 1) / T, first = u.seq / T;
        for (int b0 = 0; fine && b0 < count; b0 += kBlocks) {
            // the lane's page: entry e of the unit
            const int e = (begin + b0) * kPages + lane;
            int page = -1;
            bool old = false, young = false;
            if (b0 + lane / kPages < count && e < u.entries) {
                old = e < u.listed;
                young = sel == nullptr || !old;
                page = !old ? first + e - u.listed : sel != nullptr ? sel[e] : e;
                if (sel != nullptr && old && (page < 0 || page >= pages)) {
                    report(p.err, KVMM_ERR_OUT_OF_RANGE);
                    page = -1;
                }
            }
            int32_t phys = -1;
            if (page >= 0) {
                phys = table[page];
                if (phys < 0 || phys >= p.n_phys) {
                    report(p.err, phys < 0 ? KVMM_ERR_NULL_BLOCK : KVMM_ERR_OUT_OF_RANGE);
                    phys = -1;
                }
            }
            uint32_t settled = 0;
            int node0 = kNoNode;
            if (phys >= 0) {
                const int s = u.seq - page * T;  // settled slots of the page, when listed for them
                if (old && s > 0) settled = s >= T ? 0xffffffffu >> (32 - T) : (1u << s) - 1;
                if (young && -s < u.held && T - s > 0) node0 = -s;
            }
            const uint32_t some = __ballot_sync(kFullMask, phys >= 0);
            const uint32_t all = __ballot_sync(kFullMask, settled == 0xffffffffu >> (32 - T));
            const int blocks = min(kBlocks, count - b0);
            for (int j = 0; j < blocks; ++j) {
                const uint32_t lanes = (kPages == 32 ? kFullMask : (1u << kPages) - 1) << (j * kPages);
                const bool on = lane / kPages == j;
                const uint32_t bytes = __popc(some & lanes) * kPageBytes;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++item) {
                    const uint32_t slot = item % S::kStages;
                    fine = wait_for(&c.empty[slot], (item / S::kStages & 1) ^ 1, &c.gave_up);
                    fine = __all_sync(kFullMask, fine);
                    if (!fine) break;
                    if (kv == 0) {
                        // The slot was freed by the products of item 2 nth - kStages, which are issued after P V of
                        // block nth - kRing: nobody reads that block's masks any more.
                        BlockMask& m = c.mask[nth % kRing];
                        if (on) {
                            m.settled[mine] = settled;
                            m.node0[mine] = node0;
                        }
                        if (lane == 0) {
                            m.whole = (all & lanes) == lanes;
                            m.held = u.held;
                            m.pages = max(32 - __clz((some & lanes) >> (j * kPages)), 1);
                        }
                        ++nth;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&c.full[slot], bytes);
                    __syncwarp();
                    if (on && phys >= 0) {
                        uint8_t* dst = ring + slot * S::kTile;
                        if (kv == 0) {
#pragma unroll
                            for (int half = 0; half < D / 64; ++half)
                                tma_load_3d_hint(dst + half * (kTokens * 128) + mine * (T * 128), kmap, half * 64, 0, phys,
                                                 &c.full[slot], policy);
                        } else {
                            tma_load_3d_hint(dst + mine * kPageBytes, vmap, 0, 0, phys, &c.full[slot], policy);
                        }
                    }
                    __syncwarp();
                }
                if (!fine) break;
            }
        }
    }
    if (!fine) {  // the copies in flight land before the CTA ends
        const uint32_t n = min(item, static_cast<uint32_t>(S::kStages));
        for (uint32_t i = item - n; i < item; ++i)
            mbar_wait_bounded(&c.full[i % S::kStages], i / S::kStages & 1);
    }
}

// ---- values that nothing may see -------------------------------------------------------
// Slots of a block's values that nothing shows are set to zero: whatever they hold, NaN included, would meet a weight of
// 0.  So are nodes' values that are not finite, for the rows that do not see the node; those that do are told by `spoilt`.
// By the 128 threads of a softmax group, before they hand over the weights.
template <int D, int T>
__device__ __noinline__ void clear_unseen(uint8_t* values, const BlockMask& m, unsigned long long* spoilt)
{
    constexpr int kChunks = T / 8;
    for (int i = 0; i < m.pages; ++i) {
        uint32_t seen = m.settled[i], nodes = 0;
        const int from = max(m.node0[i], 0), to = min(m.node0[i] + T, m.held);  // its nodes (none: from >= to)
        if (from < to) nodes = ((to - from >= 32 ? 0u : 1u << (to - from)) - 1u) << (from - m.node0[i]);
        seen |= nodes;
        if (seen == 0xffffffffu >> (32 - T) && nodes == 0) continue;
        for (int x = threadIdx.x & 127; x < D * kChunks; x += 128) {
            const int d = x / kChunks, ch = x % kChunks;
            const uint32_t bits = seen >> (8 * ch) & 255u;
            const uint32_t young = nodes >> (8 * ch) & 255u;
            if (bits == 255u && young == 0) continue;
            const int at = T == 16 ? ch ^ (d >> 2 & 1) : ch ^ (d >> 1 & 3);
            uint4* q = reinterpret_cast<uint4*>(values + i * (T * D * 2) + d * (T * 2) + at * 16);
            uint4 v = *q;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                w[s] &= (bits >> (2 * s) & 1 ? 0xffffu : 0u) | (bits >> (2 * s + 1) & 1 ? 0xffff0000u : 0u);
            // (an exponent of ones carries into the sign's place)
            uint32_t wild = 0;
#pragma unroll
            for (int s = 0; s < 4; ++s) wild |= ((w[s] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
            if (wild != 0) {
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t half = s & 1 ? 0x7f800000u : 0x7f80u;
                    if ((young >> s & 1) && (w[s / 2] & half) == half) {
                        w[s / 2] &= s & 1 ? 0xffffu : 0xffff0000u;
                        atomicOr(spoilt, 1ull << (m.node0[i] + 8 * ch + s));
                    }
                }
            }
            *q = v;
        }
    }
    fence_proxy_async_shared();
}

// which of 32 channels hold a value that is not finite in any of these nodes (looked up again: hardly ever met)
template <int D, int T>
__device__ __noinline__ uint32_t spoilt_channels(const TreeAttnParams& p, const Unit& u, uint64_t nodes, int channel)
{
    uint32_t found = 0;
    for (; nodes != 0; nodes &= nodes - 1) {
        const int t = u.seq + __ffsll(static_cast<long long>(nodes)) - 1, phys = p.block_table[u.index * p.Pmax + t / T];
        const kvmm_bf16* v = p.v_pool + (static_cast<size_t>(phys) * D + channel) * T + t % T;  // (the page was copied)
        for (int e = 0; e < 32; ++e)
            if ((v[e * T] & 0x7f80u) == 0x7f80u) found |= 1u << e;
    }
    return found;
}

// ---- the issuing thread -------------------------------------------------------------
// In order: the scores of the first two steps, then, as each step's weights come, its P V and the scores of the step after
// next.  So the step of one stream has P V and Q K^T done while the other's softmax runs.  A group's scores are complete
// only when the P V before them is (its sums may then be rescaled), and they overwrite its weights behind that P V.
template <int D, int T>
__device__ void issue_products(const Launch& a, uint8_t* smem, Control& c, Walk k)
{
    using S = Smem<D>;
    constexpr uint64_t rows128 = matrix_desc(128), rowsT = matrix_desc(T * 2);
    constexpr uint32_t qk = mma_desc(128, kTokens), pv = mma_desc(128, D);
    const uint32_t base = smem_addr(smem), ring = base + 2 * S::kTile, tmem = c.tmem;
    const bool two = a.tiles == 2;
    // slot and phase of the next block's keys and of the next values: every other item of the ring
    uint32_t k_slot = 0, k_phase = 0, v_slot = 1, v_phase = 0;
    auto next = [](uint32_t& slot, uint32_t& phase) {
        slot += 2;
        if (slot >= S::kStages) {
            slot -= S::kStages;
            phase ^= 1;
        }
    };
    uint32_t piece = 0, nth = 0, p_phase = 0;  // (a bit a stream)
    bool fine = true;
    Unit u;
    int begin, count;
    while (fine && next_piece<T>(a, k, u, begin, count)) {
        fine = wait_for(&c.q_ready[0], piece & 1, &c.gave_up) && wait_for(&c.q_ready[1], piece & 1, &c.gave_up);
        tc_fence_after();
        ++piece;
        const int steps = two ? 2 * count : count;
        auto scores = [&](int v) {  // S = Q K^T of step v
            const uint32_t s = v & 1;
            const bool first = !two || s == 0, last = !two || s == 1;  // of the products that take the block's keys
            if (first && !wait_for(&c.full[k_slot], k_phase, &c.gave_up)) {
                fine = false;
                return;
            }
            const uint64_t q = matrix_at(rows128, base + s * S::kTile), kk = matrix_at(rows128, ring + k_slot * S::kTile);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint32_t off = ((i / 4) * (128 * 128) + (i % 4) * 32) >> 4;
                mma_ss(tmem + s * 128, q + off, kk + off, qk, i > 0);
            }
            mma_commit(&c.s_full[s]);
            if (last) {
                mma_commit(&c.empty[k_slot]);
                next(k_slot, k_phase);
            }
        };
        scores(0);
        if (fine && steps > 1) scores(1);
        for (int v = 0; fine && v < steps; ++v) {  // O += P V of step v
            const uint32_t s = v & 1;
            const bool first = !two || s == 0, last = !two || s == 1;
            if ((first && !wait_for(&c.full[v_slot], v_phase, &c.gave_up)) ||
                !wait_for(&c.p_ready[s], p_phase >> s & 1, &c.gave_up)) {
                fine = false;
                break;
            }
            p_phase ^= 1u << s;
            tc_fence_after();
            const uint64_t vv = matrix_at(rowsT, ring + v_slot * S::kTile);
            const uint32_t o = tmem + 256 + s * 128, w = tmem + s * 128;  // (the weights' second halves: 64 columns on)
            const int sixteens = c.mask[(nth + (two ? v >> 1 : v)) % kRing].pages * (T / 16);  // (1 at least)
#pragma unroll
            for (int i = 0; i < kTokens / 16; ++i) {
                const uint32_t off = ((i * 16 / T) * (T * D * 2) + (i * 16 % T) * 2) >> 4;
                if (i < sixteens) {
                    mma_ts(o, w + i * 8, vv + off, pv, i > 0 || (v >> 1) % kRun != 0);  // (the first of a run: not added)
                    mma_ts(o, w + 64 + i * 8, vv + off, pv, true);
                }
            }
            if (last) {
                mma_commit(&c.empty[v_slot]);
                next(v_slot, v_phase);
            }
            if (v + 2 < steps)
                scores(v + 2);
            else
                mma_commit(&c.o_done[s]);
        }
        nth += count;
    }
    if (!fine) {  // products in flight end before the CTA does
        mma_commit(&c.drain);
        mbar_wait_bounded(&c.drain, 0);
    }
}

// ---- a softmax group: the 128 threads of a stream, a row each ------------------------
// Both groups arrive and wait; false once any warp of the CTA has given up.  What either has seen done in tensor memory
// (its stream's products, its own loads and stores) is done for both behind it.
__device__ __forceinline__ bool groups_meet(Control& c, uint32_t& phase)
{
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&c.meet);
    const bool fine = wait_for(&c.meet, phase & 1, &c.gave_up);
    tc_fence_after();
    ++phase;
    return __all_sync(kFullMask, fine);
}

// row / G of a row below 512: (row / 65536 adds less than 1 / 8 to the quotient's fraction)
__device__ __forceinline__ int node_of(const TreeAttnParams& p, int row) { return row * (65536 / p.G + 1) >> 16; }

// where a row of the unit is among the nodes' heads
__device__ __forceinline__ size_t row_of(const TreeAttnParams& p, const Unit& u, int row)
{
    const int i = node_of(p, row);
    return (static_cast<size_t>(u.b) * p.n_max + i) * p.Hq + u.h * p.G + (row - i * p.G);
}

// the group's tile of queries, rows that do not exist as zeros; every load is in flight before the first store
template <int D>
__device__ __forceinline__ void load_queries(const TreeAttnParams& p, const Unit& u, int row0, uint8_t* tile)
{
    constexpr int kLoads = D / 8;
    const int t = threadIdx.x & 127, ch = t % (D / 8), r0 = t / (D / 8), end = u.row0 + u.rows;
    const kvmm_bf16* q = p.q + (static_cast<size_t>(u.b) * p.n_max * p.Hq + u.h * p.G) * D + ch * 8;
    const int magic = 65536 / p.G + 1;
    uint4 v[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
        const int row = row0 + r0 + x * (1024 / D), i = row * magic >> 16;
        v[x] = make_uint4(0, 0, 0, 0);
        if (row < end) v[x] = *reinterpret_cast<const uint4*>(q + (static_cast<size_t>(i) * p.Hq + (row - i * p.G)) * D);
    }
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
        const int r = r0 + x * (1024 / D);
        *reinterpret_cast<uint4*>(tile + (ch / 8) * (128 * 128) + r * 128 + ((ch % 8 ^ (r & 7)) << 4)) = v[x];
    }
    fence_proxy_async_shared();
}

// 32 outputs of a row
__device__ __forceinline__ void store_out32(kvmm_bf16* out, const float* o)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4*>(out)[i] =
            make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                       pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
}

// a quad of a row's sums in shared memory (see join_cluster)
template <int D>
__device__ __forceinline__ int quad_at(int row, int quad) { return row * (D / 4) + (quad ^ (row & (D / 4 - 1))); }

__device__ __forceinline__ float lse_of(float m, float l, float scale_log2)
{
    return l != 0.f ? (m * scale_log2 + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// A row's sums of a run, kRun steps: added to those of the runs before it, which are in units of 2^(before - ref) (the first
// run's are put down), or, at the end of a piece (LAST), those added to the last run's in tensor memory.
template <int D, bool LAST>
__device__ __noinline__ void carry_run(const Launch& a, uint32_t tO, float4* run, float2* kept, float ref, bool first, bool row)
{
    const float before = first || !row ? -INFINITY : kept->x;
    const float f = before == -INFINITY ? 0.f : exp2_fast((before - ref) * a.p.scale_log2);
#pragma unroll 1
    for (int i = 0; i < D / 4; i += 4) {
        uint32_t o[16];
        tmem_ld16(tO + 4 * i, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!row) continue;
            float4 x = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                   __uint_as_float(o[4 * e + 3]));
            float4* y = run + (i + e) * a.tile_rows;
            if (!first) x = make_float4(fmaf(y->x, f, x.x), fmaf(y->y, f, x.y), fmaf(y->z, f, x.z), fmaf(y->w, f, x.w));
            if (!LAST) *y = x;
            o[4 * e] = __float_as_uint(x.x);
            o[4 * e + 1] = __float_as_uint(x.y);
            o[4 * e + 2] = __float_as_uint(x.z);
            o[4 * e + 3] = __float_as_uint(x.w);
        }
        __syncwarp();
        if (LAST) tmem_st16(tO + 4 * i, o);
    }
    if (LAST) tmem_wait_st();
    if (!LAST && row) kept->x = ref;
}

template <int D, int T>
__device__ void softmax_rows(const Launch& a, uint8_t* smem, Control& c, Walk k)
{
    constexpr int kPages = kTokens / T;
    const TreeAttnParams& p = a.p;
    const int s = threadIdx.x >> 7, r = threadIdx.x & 127, warp = r >> 5, lane = r & 31;
    const bool two = a.tiles == 2;
    const uint32_t mine = c.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t tS = mine + s * 128, tO = mine + 256 + s * 128;
    const float scale = p.scale_log2, slack = 8.f / scale;
    float4* const run = a.run + static_cast<size_t>(2 * blockIdx.x + s) * (D / 4) * a.tile_rows + r;  // (not used in short units)
    uint32_t s_phase = 0, o_phase = 0, met = 0, nth = 0, piece = 0;
    Unit u;
    int begin, count;
    while (next_piece<T>(a, k, u, begin, count)) {
        // (Set before the other group's scores, which wait for both groups' queries; read last in the piece before the last one,
        // which both groups have left.)
        unsigned long long& spoilt = c.spoilt[piece++ & 1];
        if (threadIdx.x == 0) spoilt = 0;
        const int row0 = u.row0 + (two ? s * 128 : 0), row = row0 + r;
        const int rows = min(max(u.row0 + u.rows - row0, 0), 128);  // of the tile
        const bool busy = warp * 32 < rows;                          // the warp has rows
        load_queries<D>(p, u, row0, smem + s * Smem<D>::kTile);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.q_ready[s]);
        uint64_t bits = 0;
        if (r < rows) {
            const int i = node_of(p, row);
            bits = p.tree_mask != nullptr ? p.tree_mask[static_cast<size_t>(u.b) * p.n_max + i] : ~0ull >> (63 - i);
            if (u.held < 64) bits &= (1ull << u.held) - 1;
        }
        float ref = -INFINITY, l = 0.f;
        const int steps = two ? count : (count - s + 1) / 2;
        for (int v = 0; v < steps; ++v) {
            const int blk = two ? v : 2 * v + s;
            if (!__all_sync(kFullMask, wait_for(&c.s_full[s], s_phase & 1, &c.gave_up))) return;
            ++s_phase;
            tc_fence_after();
            // (the products before this block's scores are done; the meeting's place in shared memory is free until then)
            if (busy && v != 0 && v % kRun == 0) carry_run<D, false>(a, tO, run, &c.ml[s][r], ref, v == kRun, r < rows);
            if (busy) {
                uint32_t z[kTokens];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(tS + 32 * i, z + 32 * i);
                tmem_wait_ld(z);
                const BlockMask& m = c.mask[(nth + blk) % kRing];
                if (!m.whole) {
#pragma unroll
                    for (int i = 0; i < kPages; ++i) {
                        const int j = m.node0[i];  // the node in the page's first slot, below 0 where it comes later
                        uint32_t seen = m.settled[i];
                        if (j < 64 && j > -64) seen |= static_cast<uint32_t>(j >= 0 ? bits >> j : bits << -j);
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            z[i * T + t] = seen >> t & 1 ? z[i * T + t] : 0xff800000u;
                    }
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i] = __uint_as_float(z[i]);
#pragma unroll
                for (int i = 4; i < kTokens; ++i) top[i % 4] = fmaxf(top[i % 4], __uint_as_float(z[i]));
                const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                if (v == 0) {
                    ref = most;
                } else if (__any_sync(kFullMask, most > ref + slack)) {
                    // (the products before this block's scores are done: O may be changed)
                    float f = 1.f;
                    if (most > ref + slack) {
                        f = exp2_fast((ref - most) * scale);  // 0 where nothing was seen before
                        ref = most;
                        l *= f;
                    }
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + i, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                        tmem_st16(tO + i, o);
                    }
                }
                const float base = ref == -INFINITY ? 0.f : ref * scale;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kTokens / 32; ++i) {
                    uint32_t w[16], rest[16];  // two halves: what the first one's rounding (2^-8) leaves, rounded (2^-16)
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float e0 = exp2_fast(fmaf(__uint_as_float(z[32 * i + 2 * x]), scale, -base));
                        const float e1 = exp2_fast(fmaf(__uint_as_float(z[32 * i + 2 * x + 1]), scale, -base));
                        sum[(2 * x) % 4] += e0;
                        sum[(2 * x + 1) % 4] += e1;
                        w[x] = pack_bf16x2(e0, e1);
                        rest[x] = pack_bf16x2(e0 - __uint_as_float(w[x] << 16), e1 - __uint_as_float(w[x] & 0xffff0000u));
                    }
                    tmem_st16(tS + 16 * i, w);
                    tmem_st16(tS + 64 + 16 * i, rest);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
            }
            if ((!two || s == 0) && !c.mask[(nth + blk) % kRing].whole) {
                const uint32_t item = 2 * (nth + blk) + 1, slot = item % Smem<D>::kStages;
                if (!__all_sync(kFullMask, wait_for(&c.full[slot], item / Smem<D>::kStages & 1, &c.gave_up))) return;
                clear_unseen<D, T>(smem + (2 + slot) * Smem<D>::kTile, c.mask[(nth + blk) % kRing], &spoilt);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.p_ready[s]);
        }
        nth += count;
        if (steps > 0) {
            if (!__all_sync(kFullMask, wait_for(&c.o_done[s], o_phase & 1, &c.gave_up))) return;
            ++o_phase;
            tc_fence_after();
            if (busy && steps > kRun) carry_run<D, true>(a, tO, run, &c.ml[s][r], ref, false, r < rows);
        }
        // the row's result: written whole, or left as a part
        const bool whole = count == u.blocks && a.cluster <= 1;
        const size_t part = (2 * blockIdx.x + (begin > 0 ? 0 : 1)) * a.tiles + (two ? s : 0);
        float f0 = 1.f, f1 = 0.f;
        int c0 = 0, c1 = D / 32;
        const bool join = !two && count > 1;
        if (!two) {  // both streams hold the same rows: each group joins half of the channels
            c.ml[s][r] = make_float2(ref, l);
            if (!groups_meet(c, met)) return;
            const float2 other = c.ml[s ^ 1][r];
            const float m = fmaxf(ref, other.x);
            const float mine_f = l != 0.f ? exp2_fast((ref - m) * scale) : 0.f;
            const float other_f = other.y != 0.f ? exp2_fast((other.x - m) * scale) : 0.f;
            f0 = s == 0 ? mine_f : other_f;
            f1 = s == 0 ? other_f : mine_f;
            l = l * mine_f + other.y * other_f;  // (a sum is 0 only where nothing was seen: NaN goes through)
            ref = m;
            c0 = s * (D / 64);
            c1 = c0 + D / 64;
        }
        // (a cluster's CTA has one piece: behind the meeting the ring is free, and its sums go there)
        if (two && a.cluster > 1 && !groups_meet(c, met)) return;
        if (busy) {
            const float inv = l != 0.f ? 1.f / l : 0.f;
            const size_t at = r < rows ? row_of(p, u, row) : 0;
            const uint64_t wild = spoilt & bits;  // (bits of rows that do not exist are 0)
            for (int i = c0; i < c1; ++i) {
                uint32_t x[32], y[32];
                tmem_ld32(mine + 256 + (two ? s * 128 : 0) + 32 * i, x);
                tmem_ld32(mine + 384 + 32 * i, y);  // (not used unless the streams are joined)
                tmem_wait_ld(x);
                tmem_wait_ld(y);
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    o[e] = __uint_as_float(x[e]) * f0;
                    if (join) o[e] = fmaf(__uint_as_float(y[e]), f1, o[e]);
                }
                if (wild != 0) {
                    const uint32_t channels = spoilt_channels<D, T>(p, u, wild, 32 * i);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (channels >> e & 1) o[e] = __uint_as_float(0x7fc00000u);
                }
                __syncwarp();
                if (r < rows) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = l != 0.f ? o[e] * inv : 0.f;
                        store_out32(p.out + at * D + 32 * i, o);
                    } else if (a.cluster > 1) {
                        float4* dst = reinterpret_cast<float4*>(smem + 2 * Smem<D>::kTile);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[quad_at<D>(two ? s * 128 + r : r, 8 * i + e)] =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
                        float4* dst = a.o + (part * (D / 4) + 8 * i) * a.tile_rows + r;
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e * a.tile_rows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            if (r < rows && (two || s == 0)) {
                if (a.cluster > 1)
                    reinterpret_cast<float2*>(smem + 2 * Smem<D>::kTile + a.tiles * 128 * D * 4)[two ? s * 128 + r : r] =
                        make_float2(ref, l);
                else if (!whole)
                    a.ml[part * a.tile_rows + r] = make_float2(ref, l);
                else if (p.lse != nullptr)
                    p.lse[at] = lse_of(ref, l, scale);
            }
        }
        // (behind it the other stream's sums have been read, and its O)
        if (!two && !groups_meet(c, met)) return;
    }
}

// a unit to which nothing is shown: its selection is empty and its nodes have no place
__device__ __noinline__ void write_nothing(const TreeAttnParams& p, const Unit& u)
{
    for (int row = u.row0; row < u.row0 + u.rows; ++row) {
        const size_t at = row_of(p, u, row);
        for (int x = 0; x < p.D / 8; ++x) reinterpret_cast<uint4*>(p.out + at * p.D)[x] = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr) p.lse[at] = -INFINITY;
    }
}

// The CTA's run of blocks where they are dealt evenly: each thread counts some units, in order.
template <int T>
__device__ __forceinline__ void deal_blocks(const Launch& a, Control& c)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (a.units + kThreads - 1) / kThreads;
    int sum = 0;
    Unit u;
    for (int w = tid * per; w < min(a.units, (tid + 1) * per); ++w) {
        u = unit_of<T>(a, w, blockIdx.x == 0);
        sum += u.blocks;
    }
    int before = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFullMask, before, off);
        if (lane >= off) before += y;
    }
    if (lane == 31) c.sums[warp] = before;
    __syncthreads();
    int total = 0;
    before -= sum;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        const int x = c.sums[i];
        if (i < warp) before += x;
        total += x;
    }
    // Every CTA that takes part has a block: the parts of a unit come from consecutive CTAs.  CTA i begins at block
    // total * i / n, rounded down.
    const int n = min(static_cast<int>(gridDim.x), max(total, 1)), each = total / n, rest = total - each * n;
    const int cta = min(static_cast<int>(blockIdx.x), n);
    const int start = each * cta + rest * cta / n;
    const int end = cta == n ? start : each * (cta + 1) + rest * (cta + 1) / n;
    for (int w = tid * per; w < min(a.units, (tid + 1) * per); ++w) {
        if (per > 1) u = unit_of<T>(a, w, false);
        if (start < end && start >= before && start < before + u.blocks) {
            c.w0 = w;
            c.off0 = start - before;
            c.left = end - start;
            c.unit = u;
        }
        if (u.blocks == 0) {
            if (u.rows > 0 && blockIdx.x == 0) write_nothing(a.p, u);
        } else if (before >= start && before < end && before + u.blocks > end) {
            // the unit begins here and goes on, up to the CTA of its last block
            c.cut = make_int4(w, cta, static_cast<int>((static_cast<long long>(before + u.blocks) * n - 1) / total), u.rows);
        }
        if (a.by_unit && (u.blocks == 0 ? blockIdx.x == 0 : before >= start && before < end))
            a.cut[w] = u.blocks != 0 && before + u.blocks > end ? c.cut : make_int4(-1, 0, 0, 0);
        before += u.blocks;
    }
    if (a.by_unit) return;
    __syncthreads();
    if (tid == 0) a.cut[blockIdx.x] = c.cut;
}

// ---- a cluster a unit: its CTAs' sums, joined through distributed shared memory -----------
// A CTA's sums lie where its ring of blocks was: rows of D / 4 quads, a row's quads swapped by its number so that both a
// thread a row and a thread a quad reach all banks; behind them reference and sum of each row.
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t local, uint32_t rank)
{
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 ld_cluster_v2(uint32_t local, uint32_t rank)
{
    uint32_t remote;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(remote) : "memory");
    return v;
}

// K CTAs' and I quads' loads in flight: a remote one takes some 700 cycles.  (Pairs of CTAs have several quads a thread: two at
// once took eight sequences of 128 pages a head a microsecond less, four spill.)
template <int D, int K, int I>
__device__ __forceinline__ void join_quads(const Launch& a, const Unit& u, uint8_t* smem)
{
    const TreeAttnParams& p = a.p;
    const uint32_t sums = smem_addr(smem) + 2 * Smem<D>::kTile, ml = sums + a.tiles * 128 * D * 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, step = a.cluster * 256, all = u.rows * (D / 4);
    for (int x0 = (warp * a.cluster + cluster_ctarank()) * 32 + lane; x0 < all; x0 += I * step) {
        float m[I], l[I];
        float4 o[I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int k0 = 0; k0 < a.cluster; k0 += K) {
            float2 ml_k[I][K];
            float4 o_k[I][K];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int x = x0 + i * step, row = x / (D / 4), quad = x % (D / 4);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ml_k[i][k] = make_float2(-INFINITY, 0.f);
                    if (k0 + k < a.cluster && x < all) {
                        ml_k[i][k] = ld_cluster_v2(ml + row * 8, k0 + k);
                        o_k[i][k] = ld_cluster_v4(sums + quad_at<D>(row, quad) * 16, k0 + k);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float mn = m[i];
#pragma unroll
                for (int k = 0; k < K; ++k) mn = fmaxf(mn, ml_k[i][k].x);
                const float f0 = l[i] != 0.f ? exp2_fast((m[i] - mn) * p.scale_log2) : 0.f;
                m[i] = mn;
                l[i] *= f0;
                o[i] = make_float4(o[i].x * f0, o[i].y * f0, o[i].z * f0, o[i].w * f0);
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (ml_k[i][k].y != 0.f) {  // (a CTA without a block has left no sums)
                        const float f = exp2_fast((ml_k[i][k].x - mn) * p.scale_log2);
                        l[i] = fmaf(ml_k[i][k].y, f, l[i]);
                        o[i].x = fmaf(o_k[i][k].x, f, o[i].x);
                        o[i].y = fmaf(o_k[i][k].y, f, o[i].y);
                        o[i].z = fmaf(o_k[i][k].z, f, o[i].z);
                        o[i].w = fmaf(o_k[i][k].w, f, o[i].w);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int x = x0 + i * step, row = x / (D / 4), quad = x % (D / 4);
            if (x >= all) continue;
            const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
            const size_t at = row_of(p, u, u.row0 + row);
            reinterpret_cast<uint2*>(p.out + at * D)[quad] =
                make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
            if (p.lse != nullptr && quad == 0) p.lse[at] = lse_of(m[i], l[i], p.scale_log2);
        }
    }
}

template <int D>
__device__ __forceinline__ void join_cluster(const Launch& a, const Unit& u, uint8_t* smem)
{
    if (a.cluster <= 2)
        join_quads<D, 2, 2>(a, u, smem);
    else
        join_quads<D, 8, 1>(a, u, smem);
}

// ---- the kernel ---------------------------------------------------------------------
template <int D, int T>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const Launch a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using S = Smem<D>;
    Control& c = *reinterpret_cast<Control*>(smem + S::kControl);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 9) tmem_alloc_all(&c.tmem);
    if (tid == 256) {  // (the copying warp's: the maps are there before its first copy)
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.p_ready[i], 4);
            mbar_init(&c.q_ready[i], 4);
            mbar_init(&c.o_done[i], 1);
        }
        mbar_init(&c.meet, 8);
        mbar_init(&c.drain, 1);
        c.gave_up = 0;
        c.w0 = a.units;
        c.off0 = 0;
        c.left = 0;
        c.cut = make_int4(-1, 0, 0, 0);
        fence_barrier_init();
    }
    tc_fence_before();
    pdl_wait_then_release();

    if (a.cluster == 0) {
        deal_blocks<T>(a, c);
    } else if (tid == 0) {
        c.w0 = blockIdx.x / a.cluster;
        const int rank = cluster_ctarank();
        c.unit = unit_of<T>(a, c.w0, rank == 0);
        // (rounded up: the last CTA, whose last block has masks, does not get the odd blocks too)
        c.off0 = (c.unit.blocks * rank + a.cluster - 1) / a.cluster;
        c.left = (c.unit.blocks * (rank + 1) + a.cluster - 1) / a.cluster - c.off0;
        if (a.cluster == 1 && c.unit.blocks == 0 && c.unit.rows > 0) write_nothing(a.p, c.unit);
    }
    __syncthreads();
    tc_fence_after();
    const Walk k{c.w0, c.off0, c.left, &c.unit};
    // 168 registers a thread at launch: the softmax groups take 208 (a row's 128 scores stay in registers), the others 88
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        softmax_rows<D, T>(a, smem, c, k);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8)
            copy_pages<D, T>(a, &kmap, &vmap, smem, c, k);
        else if (warp == 9 && elect_one())
            issue_products<D, T>(a, smem, c, k);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.cluster > 1) {
        if (c.left == 0 && tid < a.tiles * 128)  // nothing was summed here
            reinterpret_cast<float2*>(smem + 2 * S::kTile + a.tiles * 128 * D * 4)[tid] = make_float2(-INFINITY, 0.f);
        cluster_sync();
        if (warp < 8) join_cluster<D>(a, c.unit, smem);  // (the warps that have the registers)
        cluster_sync();
    }
    if (tid == 0 && c.gave_up != 0) report(a.p.err, KVMM_ERR_TIMEOUT);
    if (warp == 9) tmem_free_all(c.tmem);
}

// ---- the parts of units that fell on several CTAs --------------------------------------
// A block takes 32 rows of a unit, a lane a row.  With many parts a unit (SLICES = 4) its warps share them, and the block
// takes 32 channels; with few, each warp takes D / 8 channels over all parts.
constexpr int kJoinWarps = 8;

template <int D, int SLICES>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const Launch a)
{
    constexpr int Q = SLICES == 1 ? D / 32 : 4;  // quads of a warp
    __shared__ float4 other[SLICES > 1 ? kJoinWarps : 1][Q][32];
    __shared__ float2 sums[kJoinWarps][32];
    const TreeAttnParams& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = warp % SLICES, quad0 = (blockIdx.z * (kJoinWarps / SLICES) + warp / SLICES) * Q;
    pdl_wait_then_release();
    const int4 cut = a.cut[blockIdx.x];
    const int row = blockIdx.y * 32 + lane, first = cut.y, last = cut.z, rows = cut.w;
    if (cut.x < 0 || blockIdx.y * 32 >= rows) return;
    const int tile = row >> 7, r = min(row & 127, a.tile_rows - 1);  // (a lane without a row reads what lies there)
    auto part = [&](int cta) { return static_cast<size_t>(2 * cta + (cta == first ? 1 : 0)) * a.tiles + tile; };
    constexpr int kAhead = Q > 2 ? 2 : 4;  // parts whose loads are in flight
    float m = -INFINITY, l = 0.f;
    float4 o[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int cta0 = first + slice; cta0 <= last; cta0 += kAhead * SLICES) {
        float2 ml[kAhead];
        float4 y[kAhead][Q];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int cta = cta0 + k * SLICES;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (cta <= last) {
                ml[k] = a.ml[part(cta) * a.tile_rows + r];
                const float4* x = a.o + (part(cta) * (D / 4) + quad0) * a.tile_rows + r;
#pragma unroll
                for (int i = 0; i < Q; ++i) y[k][i] = x[i * a.tile_rows];
            }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) mn = fmaxf(mn, ml[k].x);
        const float f0 = l != 0.f ? exp2_fast((m - mn) * p.scale_log2) : 0.f;
        m = mn;
        l *= f0;
#pragma unroll
        for (int i = 0; i < Q; ++i) o[i] = make_float4(o[i].x * f0, o[i].y * f0, o[i].z * f0, o[i].w * f0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (ml[k].y == 0.f) continue;
            const float f = exp2_fast((ml[k].x - m) * p.scale_log2);
            l = fmaf(ml[k].y, f, l);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                o[i].x = fmaf(y[k][i].x, f, o[i].x);
                o[i].y = fmaf(y[k][i].y, f, o[i].y);
                o[i].z = fmaf(y[k][i].z, f, o[i].z);
                o[i].w = fmaf(y[k][i].w, f, o[i].w);
            }
        }
    }
    if (SLICES > 1) {
#pragma unroll
        for (int i = 0; i < Q; ++i) other[warp][i][lane] = o[i];
        sums[warp][lane] = make_float2(m, l);
        __syncthreads();
        if (slice != 0) return;
        float most = m;
#pragma unroll
        for (int k = 1; k < SLICES; ++k) most = fmaxf(most, sums[warp + k][lane].x);
        const float f0 = l != 0.f ? exp2_fast((m - most) * p.scale_log2) : 0.f;
        m = most;
        l *= f0;
#pragma unroll
        for (int i = 0; i < Q; ++i) o[i] = make_float4(o[i].x * f0, o[i].y * f0, o[i].z * f0, o[i].w * f0);
#pragma unroll
        for (int k = 1; k < SLICES; ++k) {
            const float2 ml = sums[warp + k][lane];
            if (ml.y == 0.f) continue;
            const float f = exp2_fast((ml.x - m) * p.scale_log2);
            l = fmaf(ml.y, f, l);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float4 y = other[warp + k][i][lane];
                o[i] = make_float4(fmaf(y.x, f, o[i].x), fmaf(y.y, f, o[i].y), fmaf(y.z, f, o[i].z), fmaf(y.w, f, o[i].w));
            }
        }
    }
    if (row >= rows) return;
    const int bh = cut.x >> (a.groups - 1), b = bh / p.Hkv, g = cut.x & (a.groups - 1);
    Unit u;
    u.b = a.b0 + b;
    u.h = bh - b * p.Hkv;
    const size_t at = row_of(p, u, g * a.tiles * 128 + row);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint2* out = reinterpret_cast<uint2*>(p.out + at * D) + quad0;
#pragma unroll
    for (int i = 0; i < Q; ++i)
        out[i] = make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
    if (p.lse != nullptr && quad0 == 0) p.lse[at] = lse_of(m, l, p.scale_log2);
}

// most pages of a unit: all, or the selected ones and those that nodes reach
long long pages_of(int Pmax, int Kmax, int n_max, int T, bool selected)
{
    return selected ? static_cast<long long>(Kmax) + (n_max + T - 2) / T + 1 : Pmax;
}

long long blocks_of(long long pages, int T) { return (pages * T + kTokens - 1) / kTokens; }

// rows of the nodes' tiles, and how the units are cut
struct Cut {
    int tiles, groups, tile_rows, batches;  // batches: of one launch
    bool runs;  // a stream may have more than kRun steps
    Cut(int n_max, int G, int Hkv, int B, int T, int Pmax, int Kmax)
    {
        const int rows = n_max * G;
        tiles = rows > 128 ? 2 : 1;
        groups = (rows + 128 * tiles - 1) / (128 * tiles);
        tile_rows = rows < 128 ? rows : 128;
        batches = kUnitsAtOnce / (Hkv * groups);
        batches = batches < 1 ? 1 : batches > B ? B : batches;
        const long long all = pages_of(Pmax, Kmax, n_max, T, false), some = pages_of(Pmax, Kmax, n_max, T, true);
        runs = blocks_of(all > some ? all : some, T) * tiles > 2 * kRun;
    }
    static constexpr size_t kCutBytes = (sizeof(int4) * kTreeMaxCtas + 255) / 256 * 256;
    size_t rows() const { return static_cast<size_t>(2 * kTreeMaxCtas) * tiles * tile_rows; }
    size_t ml_bytes() const { return round256(sizeof(float2) * rows()); }
    size_t o_bytes(int D) const { return sizeof(float) * rows() * D; }
    size_t run_bytes(int D) const { return runs ? sizeof(float) * 2 * kTreeMaxCtas * tile_rows * D : 0; }
};

constexpr int kMaxCluster = 16;

// clusters of c CTAs of this kernel that the device holds at once
int clusters_at_once(void (*kernel)(Launch, CUtensorMap, CUtensorMap), size_t smem, int c)
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
        return -1;
    }
    return n > 0 ? n : -1;
}

template <int D, int T>
cudaError_t launch(const TreeAttnParams& p, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    struct Device {
        int dev = -1, sms = 0;
        int held[17] = {};  // clusters of c CTAs held at once; 0: not asked yet, -1: none
    };
    static thread_local Device known;  // per thread and kernel
    if (known.dev != dev) {
        known = Device{};
        e = cudaFuncSetAttribute(tree_attn_kernel<D, T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(tree_attn_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Smem<D>::kBytes));
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&known.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known.dev = dev;
    }
    CUtensorMap kmap, vmap;
    const uint64_t n = static_cast<uint64_t>(p.n_phys < INT32_MAX ? p.n_phys : INT32_MAX);
    e = tensor_map_3d(&kmap, p.k_pool, D, T, n, 64, T, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    e = tensor_map_3d(&vmap, p.v_pool, T, D, n, T, D, T == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;

    const Cut cut(p.n_max, p.G, p.Hkv, p.B, T, p.Pmax, p.Kmax);
    Launch a{};
    a.p = p;
    a.tiles = cut.tiles;
    a.groups = cut.groups;
    a.tile_rows = cut.tile_rows;
    char* ws = static_cast<char*>(p.workspace);
    a.cut = reinterpret_cast<int4*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + Cut::kCutBytes);
    a.o = reinterpret_cast<float4*>(ws + Cut::kCutBytes + cut.ml_bytes());
    a.run = cut.runs ? a.o + cut.o_bytes(D) / sizeof(float4) : nullptr;
    const long long most = blocks_of(pages_of(p.Pmax, p.Kmax, p.n_max, T, p.sel_idx != nullptr), T);  // blocks of a unit
    const int rows = p.n_max * p.G < 128 * cut.tiles ? p.n_max * p.G : 128 * cut.tiles;
    for (a.b0 = 0; a.b0 < p.B; a.b0 += cut.batches) {
        a.nb = p.B - a.b0 < cut.batches ? p.B - a.b0 : cut.batches;
        a.units = a.nb * p.Hkv * cut.groups;
        // A cluster a unit, of the most CTAs whose clusters all run at once (7 of 16, 8 of 12, 15 of 9), where units are short:
        // no second launch, and no CTA looks through all units for its own.  Beyond that the SMs that whole clusters leave
        // empty, and waiting for the longest of ragged sequences, cost more; so do clusters of more than ten CTAs of two
        // tiles, which have most to join.  Clusters against dealing (us; tables of the sequences' length), 8 KV heads of 4
        // query heads, trees of 8: one sequence of 4K tokens 13.6, 16.0, of 12K 21.3, 22.9, of 24K (193 blocks) 33.2, 30.0;
        // two of 8K 24.0, 27.5, of 16K 39.5, 36.8; four of 8K 33.3, 37.1; sixteen of 2K 31.9, 39.6; sixteen ragged ones of up
        // to 16K, 13 nodes x 5 heads 167, 134.  Two tiles, trees of 64: two of 4K (clusters of 9) 28.0, 30.0, four of 4K 35.1,
        // 40.6, of 8K (65 blocks) 53.0, 56.6; clusters of 12 and dealing, one of 2K 18.9, 17.8, of 4K 21.3, 21.3, of 8K 27.6,
        // 25.9.  The rule misses one of 1K (9 blocks, clusters of 9): 18.6, 16.2.
        int c = 0;
        if (a.units <= known.sms) {
            c = 1;
            for (int k = 2; k <= kMaxCluster && k <= most && a.units * k <= known.sms; ++k) {
                int& held = known.held[k];
                if (held == 0) held = clusters_at_once(tree_attn_kernel<D, T>, Smem<D>::kBytes, k);
                if (held >= a.units) c = k;
            }
        }
        a.cluster = c > 0 && most * cut.tiles <= kShort && c * cut.tiles <= 20 ? c : 0;
        if (a.cluster > 0) {
            e = launch_pdl_cluster(tree_attn_kernel<D, T>, dim3(static_cast<unsigned>(a.units * c)), dim3(kThreads),
                                   Smem<D>::kBytes, stream, static_cast<unsigned>(c), a, kmap, vmap);
            if (e != cudaSuccess) return e;
            continue;
        }
        long long ctas = most * a.units;
        if (ctas > known.sms) ctas = known.sms;
        if (ctas > kTreeMaxCtas) ctas = kTreeMaxCtas;
        a.by_unit = a.units <= ctas;
        e = launch_pdl(tree_attn_kernel<D, T>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Smem<D>::kBytes, stream, a,
                       kmap, vmap);
        if (e != cudaSuccess) return e;
        if (ctas == 1) continue;  // nothing is cut
        const unsigned at = static_cast<unsigned>(a.by_unit ? a.units : ctas), groups32 = (rows + 31) / 32;
        if (ctas > 4ll * a.units)
            e = launch_pdl(tree_join_kernel<D, 4>, dim3(at, groups32, D / 32), dim3(kJoinWarps * 32), 0, stream, a);
        else
            e = launch_pdl(tree_join_kernel<D, 1>, dim3(at, groups32), dim3(kJoinWarps * 32), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t tree_ws_bytes(const kvmm_shape& s, int n_max)
{
    const Cut cut(n_max, s.Hq / s.Hkv, s.Hkv, s.B, s.T, s.Pmax, s.Kmax);
    return Cut::kCutBytes + cut.ml_bytes() + cut.o_bytes(s.D) + cut.run_bytes(s.D);
}

cudaError_t launch_tree_attention(const TreeAttnParams& p, cudaStream_t stream)
{
    if (p.D == 128) return p.T == 16 ? launch<128, 16>(p, stream) : launch<128, 32>(p, stream);
    return p.T == 16 ? launch<64, 16>(p, stream) : launch<64, 32>(p, stream);
}

}  // namespace kvmm
