// paged_attn.cuh -- the kernel of attention of new tokens over a paged key/value
// cache on sm_103a, for ordinary batches (paged.cu) and for batches whose sequences
// share their first pages (prefix.cu).
//
//     O = softmax(scale q K^T + mask) V,  LSE,  per (new token, query head),
// with K and V of a sequence in pages of 16 .. 256 keys.  One kernel for every
// case, from one token of one sequence to chunks of thousands: the query heads
// that share a KV head and up to 128 / group tokens form the 128 rows of a
// tile, so a KV head's pages are read once per tile, not once per head.
//
// Bounds: with few rows per KV head (single tokens) the pages' bytes over HBM;
// with many, the chain scores -> softmax -> P.V of each 128 x 128 block, whose
// products alone take about 1000 cycles at d = 128 and which now takes about 1400,
// and under sustained load the power limit (1380 W, SM clock 1.8 of 2.07 GHz).  The
// tile is M = 128 in both: with 8 live rows the padded products still take less
// time than the block's 64 KB take to arrive at one SM's share of HBM (about 2700
// cycles), and warps without a live row skip the softmax.  Measured on one GB300:
//   one new token, 64/8 heads of 128, one sequence of 131072 keys   88 us (6.1 TB/s)
//   the same for 64 sequences of up to 8192 keys                   203 us (6.5 TB/s)
//   2048 new tokens over 8192 keys, 64/8 heads of 128              336 us in a loop,
//                              300 us before the power limit (1.43 / 1.6 PFLOP/s)
//   8 sequences, up to 500 new tokens over 4001 keys, 16 heads of 160   66 us
//   one new token over 500 keys                                     11 us in a graph
//
// Persistent, one CTA per SM.  The work is cut into equal shares of blocks, or
// handed out in whole tiles (paged_sched.cuh).  Structure (384 threads):
//   warp 3  scheduler: the CTA's next segments (tiles, or pieces of them), in a ring
//           of jobs that the others read
//   warp 0  K, by TMA: one box per page and column chunk; and each tile's Q
//   warp 2  V, into its own ring; rows past the sequence's end are zeroed in
//           shared memory, so that what the page holds there (NaN included)
//           meets no product
//   warp 1  issues the tcgen05 MMAs: S_j = Q K_j^T into one of two TMEM score
//           buffers, then O += P_{j-1} V_{j-1} with P read from TMEM
//   warps 4-11  online softmax, one row per TMEM lane, two column halves of 64
//           keys; for d <= 128 each half keeps its own maximum, sum and O
//           accumulator, merged at the tile's end; for d = 160 TMEM has room
//           for one accumulator and the halves exchange their block maxima
// Probabilities are rounded to bf16 for the product (the row sum is taken
// before; tiles of few rows carry the remainder along, kFineRows), everything else
// is fp32; the running maximum moves only when it grows by more than 2^8.
//
// A whole tile's rows go to O; a cut tile's parts go to the workspace as fp32
// rows divided by their own sum, with their own base-2 LSE, and a second kernel
// joins them: O = sum_p w_p O_p / sum_p w_p, w_p = 2^(lse_p - max).
#pragma once
#include <stddef.h>

#include <type_traits>

#include "kernels.h"
#include "paged_sched.cuh"
#include "prefix_plan.cuh"
#include "ptx.cuh"
#include "tile.cuh"

namespace ac {

namespace {

// Tiles of at most this many rows are bound by their keys' bytes, with the tensor core
// idle most of the time.  In batches of such tiles (single tokens) P goes in as two bf16
// terms, the rounded value and what the rounding left, so that only O's own rounding is
// left of the error: 1.7e-3 in the 2-norm, against 2.3e-3 with P rounded.  Measured: 64
// sequences to 8192 keys 200 -> 206 us, one of 131072 keys 87 -> 89, one of 500 keys
// 9.6 -> 10.6 in a graph (few blocks, one after another: their longer chain shows).  A
// kernel of its own: the choice inside the loop cost the others 3 to 4%.
constexpr int kFineRows = 32;
inline bool fine_batch(const PagedArgs& a) { return (int64_t)a.t.n_tokens * a.group <= (int64_t)kFineRows * a.t.n_seq; }
constexpr int kPagedMaxCtas = 160;   // workspace slots; a GB300 has 152 SMs

// Layout of a [ROWS x D] tile of Q, K or V: column chunks of 64 with the 128-byte
// swizzle, then, for D = 96 and 160, one of 32 with the 64-byte swizzle.  (Chunks
// of 32 throughout, as the core's tiles have, cost 5 TMA boxes a page instead of
// 3 at D = 160, and small boxes bound the loads: about 40 cycles each.)
template <int D, int ROWS = 128>
struct PagedGeom {
    static constexpr int WIDE = D / 64;                       // chunks of 64 columns
    static constexpr bool NARROW = D % 64 != 0;               // and one of 32
    static constexpr int CHUNKS = WIDE + (NARROW ? 1 : 0);
    static constexpr uint32_t TILE = (uint32_t)ROWS * D * 2;
    static constexpr uint32_t WIDE_BYTES = ROWS * 128, OFF_NARROW = WIDE * WIDE_BYTES;
    static_assert(D % 32 == 0 && (!NARROW || D % 64 == 32), "head dimension");
    __host__ __device__ static constexpr bool narrow(int ch) { return ch >= WIDE; }
    __host__ __device__ static constexpr uint32_t offset(int ch) { return (uint32_t)ch * WIDE_BYTES; }
    __host__ __device__ static constexpr uint32_t row_bytes(int ch) { return narrow(ch) ? 64 : 128; }
    // K-major operand: the 16-wide slice kk of the head dimension
    __device__ static __forceinline__ uint64_t desc_k(uint32_t base, int kk)
    {
        if (kk < 4 * WIDE)
            return desc_plus(smem_desc(base, 16, 1024, 2u), ((kk / 4) * WIDE_BYTES + (kk % 4) * 32) >> 4);
        return desc_plus(smem_desc(base + OFF_NARROW, 16, 512, 4u), ((kk - 4 * WIDE) * 32) >> 4);
    }
    // MN-major operand: rows [16 kk, 16 kk + 16) as the reduction slice, the wide
    // columns (or the narrow chunk's) as N
    __device__ static __forceinline__ uint64_t desc_wide(uint32_t base, int kk)
    {
        return desc_plus(smem_desc(base, WIDE_BYTES, 1024, 2u), (uint32_t)(kk * 16 * 128) >> 4);
    }
    __device__ static __forceinline__ uint64_t desc_narrow(uint32_t base, int kk)
    {
        return desc_plus(smem_desc(base + OFF_NARROW, ROWS * 64, 512, 4u), (uint32_t)(kk * 16 * 64) >> 4);
    }
};

template <int D, bool PREFIX = false>
struct PagedCfg {
    using G = TileGeom<D>;                                    // the O stage
    static constexpr uint32_t TILE = PagedGeom<D>::TILE;
    static constexpr uint32_t CHUNK = G::template chunk_bytes<128>();
    // One Q buffer (the next tile's Q loads behind this tile's last softmax and
    // epilogue), K and V rings, and for d <= 128 a stage through which a full
    // tile's O leaves by TMA.
    static constexpr int NQ = (D <= 64) ? 2 : 1;
    static constexpr int SK = (D <= 64) ? 6 : (D <= 96 ? 4 : (D <= 128 ? 3 : 2));
    static constexpr int SV = (D <= 64) ? (PREFIX ? 4 : 5) : (D <= 96 ? 3 : 2);
    static constexpr bool STAGE_O = D <= 128 && !PREFIX;
    static constexpr bool SPLIT = (D <= 128);
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = NQ * TILE;
    static constexpr uint32_t OFF_V = OFF_K + SK * TILE;
    static constexpr uint32_t OFF_OST = OFF_V + SV * TILE;
    // batches of shared pages: rows are turned over there on their way to the workspace (2 KB
    // a warp), and the plan
    static constexpr uint32_t OFF_TURN = OFF_OST, OFF_PLAN = OFF_TURN + 8 * 2048;
    static constexpr uint32_t OFF_BAR =
        PREFIX ? OFF_PLAN + ((uint32_t)sizeof(PlanNear) + 127) / 128 * 128 : OFF_OST + (STAGE_O ? TILE : 0);
    static constexpr uint32_t BAR_BYTES = 1024;
    static constexpr uint32_t OFF_XCH = OFF_BAR + BAR_BYTES;
    static constexpr uint32_t XCH_BYTES = SPLIT ? 128 * 8 : 0;
    static constexpr uint32_t SMEM = OFF_XCH + XCH_BYTES + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
    static constexpr uint32_t T_S0 = 0, T_S1 = 128, T_O = 256, T_O1 = 256 + D, T_X = 256 + D;
    static_assert(SPLIT ? (T_O1 + D <= 512) : (T_X + 6 <= 512), "TMEM budget");
};

// What a block of 128 keys and 128 rows costs a processor, in units of the kernel for few
// rows (64 keys), by which the two kernels share the processors.  Taken by measurement, one
// for all head dimensions: with 2, 3 and 4 the 64 samples take 49, 50 and 57 us, the long
// document 108, 108 and 134, drafts (d = 160) 31, 30 and 30, 64 samples at d = 64 43, 42 and
// 40, 32 samples of 20000 keys at d = 96 35, 38 and 39, 16 sequences of 40 tokens 74, 79 and 79.
constexpr int64_t kManyUnitCost = 2;
__device__ __forceinline__ int64_t many_ctas(int64_t many, int64_t few, int64_t ctas)
{
    const int64_t n = few > 0 ? quot(ctas * kManyUnitCost * many, kManyUnitCost * many + few) : ctas;
    return n > 0 ? n : 1;
}

constexpr int kJobs = 4;
// Barriers of block g's ring slots (g % SK for K, g % SV for V) serve every role that
// waits for the same event, so each product is committed once: s_full (S_g is in TMEM;
// K's slot is free) and pv_done (O has block g; V's slot and the score buffer with P
// are free).
struct PagedBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[6], v_full[6], s_full[6], pv_done[6];
    uint64_t v_tail;        // a tile's last, partial V block has landed (rows past its end still to be zeroed)
    uint64_t drain;         // every product is done (before TMEM is released)
    uint64_t never;
    // completed by all row threads
    uint64_t p_full[2][2];  // [part][score buffer] P of the part (32 keys of each half) is in TMEM
    uint64_t xmax[2];       // d = 160: row-max exchange between the column halves
    uint64_t lsum, lsum2;   // row-statistics exchange at the end of a tile
    uint64_t o_free;        // the tile's O has been read
    uint64_t ost_full;      // a full tile's O is in the stage
    uint64_t job_empty[kJobs];   // every consumer has read the job
    uint64_t job_full[kJobs];
    int64_t warp_sum[kThreads / 32], warp_tiles[kThreads / 32];
    SegmentWalk walk;       // where this CTA's share starts
    uint32_t tmem_base;
    int32_t abort_flag;
    Segment job[kJobs];     // what the scheduling warp hands to the others
};
constexpr int kJobReaders = 3 + kRowThreads / 32;              // warps: K, V, MMA and the rows
constexpr int kBarsOnce = offsetof(PagedBars, p_full) / 8;     // one arrival (a commit or a producer)
constexpr int kBarsRows = offsetof(PagedBars, job_empty) / 8;  // kRowThreads
static_assert(sizeof(PagedBars) <= PagedCfg<64>::BAR_BYTES, "barrier block");

enum : int32_t {
    kSiteInject = 1, kSiteJobEmpty, kSiteJobFull, kSiteKEmpty, kSiteVEmpty, kSiteQEmpty, kSiteQFull, kSiteKFull,
    kSiteVFull, kSiteVTail, kSitePFull, kSiteSFull, kSitePvDone, kSiteXmax, kSiteOFree, kSiteLsum, kSiteStage,
    kSiteDrain
};
__device__ __forceinline__ int32_t timeout_code(int32_t site) { return 6 | (site << 8); }

// A whole warp's bounded wait, in few instructions where the phase is complete
// already: the issuing warp's loop has to stay small (its instructions are
// fetched between those of the row warps), so the waiting itself is out of line.
// Not for the row warps, whose registers a call would spill.
static __device__ __noinline__ bool wait_longer(volatile int* abort_flag, int32_t* status, uint64_t timeout_ns,
                                                uint32_t bar, uint32_t parity, int32_t code)
{
    const WaitCtx w{abort_flag, status, timeout_ns};
    return __all_sync(0xffffffffu, wait_bounded<true>(w, bar, parity, code));
}
__device__ __forceinline__ bool wait_w(const WaitCtx& w, uint32_t bar, uint32_t parity, int32_t code)
{
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_longer(w.abort_flag, w.status, w.timeout_ns, bar, parity, code));
}

// TMA loads issued by whole warps: called converged by all 32 lanes, elect.sync
// picks the one that issues.  The operands stay in warp-uniform code: 15 to 28
// cycles a load, against 53 when a lane per page issues its own and 65 from
// inside an `if (lane == 0)` (16 loads of 2 KB from one warp).
__device__ __forceinline__ void tma_load_3d_warp(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_warp(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                                                 uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* tm, uint32_t src, int x, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
        ::"l"(reinterpret_cast<uint64_t>(tm)), "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// What the join needs to know of a cut tile, written by the CTA that has its
// first part (slot 1 of its own two; the later parts are in slot 0 of the CTAs
// after it).
struct CutTile {
    int32_t last_cta;    // 0: this CTA cut no tile at its end
    int32_t q_tok, n_rows, head;
};

// Workspace: parts [CTA][slot] of 128 fp32 rows, their base-2 LSEs, CutTile [CTA].
__host__ __device__ inline size_t part_row(int cta, int slot) { return ((size_t)cta * 2 + slot) * 128; }
__host__ __device__ inline size_t ws_lse_offset(int d) { return (size_t)kPagedMaxCtas * 2 * 128 * d * sizeof(float); }
__host__ __device__ inline size_t ws_cut_offset(int d)
{
    return ws_lse_offset(d) + (size_t)kPagedMaxCtas * 2 * 128 * sizeof(float);
}

// Batches of shared pages: behind the parts come whole tiles' rows that another tile's
// are joined with (two sets of n_tokens x h_q, of the sequences' own keys and of the
// groups'), and a record per (set, new token, head) says where the row lies.
__host__ __device__ inline size_t whole_row(const PagedTables& t, bool prefix, int tok, int head)
{
    return (size_t)kPagedMaxCtas * 2 * 128 + ((size_t)(prefix ? t.n_tokens : 0) + tok) * t.h_q + head;
}
__host__ __device__ inline size_t record_at(const PagedTables& t, bool prefix, int tok, int head)
{
    return ((size_t)(prefix ? t.n_tokens : 0) + tok) * t.h_q + head;
}
constexpr uint64_t kRecordNone = 0, kRecordWhole = 1, kRecordCut = 2, kRecordState = 3, kRecordJoined = 4,
                   kRecordFew = 8;
// `row`: its row in its tile; of a cut tile, who has its first and
// its last part (CTAs here, warps of the kernel for few rows, kRecordFew)
__device__ __forceinline__ uint64_t make_record(bool whole, bool joined, int first, int last, int row)
{
    return (whole ? kRecordWhole : kRecordCut) | (joined ? kRecordJoined : 0) | (uint64_t)row << 4 |
           (uint64_t)first << 12 | (uint64_t)last << 32;
}

// Position in a ring of N slots: the slot, and the parity of its current use.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance()
    {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

__host__ __device__ inline size_t ws_counter_offset(int d)
{
    return (ws_cut_offset(d) + kPagedMaxCtas * sizeof(CutTile) + 255) & ~(size_t)255;
}

// A value that all lanes of a warp hold alike, in a form that the compiler knows to
// be warp-uniform.  The producing and issuing warps' operands (descriptors,
// coordinates, barriers) then live in uniform registers; from ordinary ones each
// TMA load or product pays for moving its operands over (88 cycles a load, 40 a
// product, against 28 and 23).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Which split (paged_sched.cuh) a batch gets: `tiles` tiles of `units` blocks in all,
// in `heads` pairs of a sequence and a KV head, over `ctas` CTAs.  Whole tiles want
// enough of them to go round (fewer than 1.4 a CTA leave CTAs without work), several
// per KV head (or they bring nothing).  Then they win while they are few, by the parts
// that need no join, and beyond that where the keys do not fit L2 and would be read
// again for each row tile.  Measured, cut shares against whole tiles:
//   336 tiles, 174 MB of keys and values, d = 160      88 -> 66 us
//   512 tiles, 262 MB                                 171 -> 113
//   536 tiles, 356 MB, 8 heads a KV head              211 -> 143
//   296 tiles, 87 MB, d = 160                          70 -> 64
//   256 tiles, 17 MB, one sequence                     39 -> 39
// and with the counter set on both sides (the launcher leaves it out where these sizes
// cannot gain):
//   272 tiles of 5 blocks, 40 MB                       33 -> 29
//   1024 tiles, 34 MB                                 309 -> 313
//   512 tiles of 2.5 blocks, 33 MB                     27 -> 29
//   256 tiles, one per head, 333 MB                    67 -> 73
constexpr int64_t kManyBytes = 100000000;   // what L2 (129 MB) holds of them beside Q, O and the parts
__device__ __forceinline__ bool hand_out_tiles(int64_t units, int64_t tiles, int64_t heads, int64_t ctas, int d)
{
    if (10 * tiles < 14 * ctas || 2 * tiles < 3 * heads) return false;
    if (2 * tiles <= 5 * ctas) return true;
    // bytes of the keys and values, whose blocks each head's tiles visit again
    return quot(units * heads, tiles) * (128 * 4 * d) > kManyBytes;
}

// A reader's side of the jobs: false at the end (or on a wait that ran out).
template <bool SPECIAL, bool PREFIX>
__device__ __forceinline__ bool next_job(PagedBars* bars, const WaitCtx& wc, Ring<kJobs>& jr, Segment& g)
{
    const uint32_t full = smem_u32(&bars->job_full[jr.slot]);
    if constexpr (SPECIAL) {
        if (!wait_w(wc, full, jr.phase, timeout_code(kSiteJobFull))) return false;
        const Segment& s = bars->job[jr.slot];
        g.seq = uniform(s.seq);
        g.head = uniform(s.head);
        g.q_tok = uniform(s.q_tok);
        g.n_tok = uniform(s.n_tok);
        g.kv = uniform(s.kv);
        g.j0 = uniform(s.j0);
        g.j1 = uniform(s.j1);
        if constexpr (PREFIX) g.m = uniform(s.m);
    } else {
        if (!wait_warp(wc, full, jr.phase, timeout_code(kSiteJobFull))) return false;
        g = bars->job[jr.slot];
    }
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&bars->job_empty[jr.slot]));
    jr.advance();
    return g.j0 >= 0;
}
// The next one with blocks to visit, for the producing and issuing warps (the others
// only have zeros to write, which is the row threads' business).
template <bool PREFIX>
__device__ __forceinline__ bool next_work(PagedBars* bars, const WaitCtx& wc, Ring<kJobs>& jr, Segment& g)
{
    while (next_job<true, PREFIX>(bars, wc, jr, g))
        if (g.j1 > g.j0) return true;
    return false;
}

}  // namespace

// FINE: tiles of at most kFineRows rows carry P in two terms, and those of a group's shared
// keys, whose rows would be such tiles' one by one.
// PREFIX: the sequences are a plan's (PrefixSeq), whose rows may have their keys in two
// of them; such rows go to the workspace, and records say where each row's parts lie.
template <int D, bool FINE, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedArgs a)
{
    using G = TileGeom<D>;
    using P = PagedGeom<D>;
    using C = PagedCfg<D, PREFIX>;
    const PagedTables& t = a.t;
    using Tables = std::conditional_t<PREFIX, PrefixTables, PagedTables>;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    Tables tab;
    if constexpr (PREFIX)
        tab = PrefixTables{a.plan ? a.plan : reinterpret_cast<const PlanNear*>(smem_raw + pad + C::OFF_PLAN)->seq, a.n_plan,
                           t.h_kv};
    else
        tab = t;
    const uint32_t sb = raw + pad;
    PagedBars* bars = reinterpret_cast<PagedBars*>(smem_raw + pad + C::OFF_BAR);
    auto bar = [](uint64_t& b) { return smem_u32(&b); };
    const uint32_t warp = (uint32_t)uniform((int)warp_id()), lane = lane_id();

    // Set-up, spread over the warps: warp 3 the barriers, warp 1 TMEM, warp 0 the
    // descriptors, and from warp 4 on the lengths.
    if (warp == 3) {
        uint64_t* all = reinterpret_cast<uint64_t*>(bars);
        for (int i = lane; i < kBarsRows; i += 32) mbar_init(bar(all[i]), i < kBarsOnce ? 1 : kRowThreads);
        if (lane < kJobs) {
            mbar_init(bar(bars->job_empty[lane]), kJobReaders);
            mbar_init(bar(bars->job_full[lane]), 1);
        }
        if (lane == 0) {
            bars->abort_flag = 0;
            if constexpr (!PREFIX) reinterpret_cast<CutTile*>(a.ws + ws_cut_offset(D))[blockIdx.x].last_cta = 0;
        }
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < (P::NARROW ? 2 : 1); ++i) {
            tma_prefetch_desc(&maps.q[i]);
            tma_prefetch_desc(&maps.k[i]);
            tma_prefetch_desc(&maps.v[i]);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }

    // the plan is another kernel's, this one's set-up so far runs beside it
    if constexpr (PREFIX) {
        PlanNear* near = reinterpret_cast<PlanNear*>(smem_raw + pad + C::OFF_PLAN);
        // the kernel for few rows, which starts beside this one, goes by what CTA 0 says
        // (plan_written)
        auto say = [&](uint64_t what) {
            if (blockIdx.x == 0 && threadIdx.x == 0)
                asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.stamp_at), "l"(a.stamp + what) : "memory");
        };
        if (a.plan) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            say(1);
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            __syncthreads();
        } else {
            say(0);
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            prefetch_table(t);
            plan_near(t, a.tpt, a.causal, a.groups, *near);
            if (blockIdx.x == 0) {
                for (int i = threadIdx.x; i < a.n_plan; i += kThreads) a.plan_out[i] = near->seq[i];
                if (threadIdx.x == 0) *a.many_units = (int64_t)near->many;
                __syncthreads();
                say(1);
            }
        }
        // CTAs without a share make room at once for the kernel for few rows
        const int64_t many = a.plan ? *a.many_units : (int64_t)near->many;
        if ((many == 0 || (int64_t)blockIdx.x >= many_ctas(many, tab.plan[a.n_plan - 1].few_units, gridDim.x)) &&
            !a.inject_timeout) {
            tc_fence_after();
            if (warp == 1) tmem_dealloc(bars->tmem_base, 512);
            return;
        }
    }

    // ---- this CTA's share of the line: every thread sums the units of its run of
    // sequences, the block sums those, and the warp whose runs hold the share's first
    // unit finds its tile.
    const int order = ((int)threadIdx.x + kThreads - 128) % kThreads;     // warp 4 first
    const int run = (tab.n_seq + kThreads - 1) / kThreads;
    const int s0 = order * run < tab.n_seq ? order * run : tab.n_seq;
    const int s1 = s0 + run < tab.n_seq ? s0 + run : tab.n_seq;
    int64_t mine = 0, mine_tiles = 0, mine_heads = 0;
    int per_head = 0;
    SeqTable table{};
    for (int s = s0; s < s1; ++s) {
        table = read_seq(tab, s, a.tpt, a.causal);
        if (table.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
        per_head = table.s.units(table.s.tiles());
        mine += (int64_t)per_head * t.h_kv;
        mine_tiles += (int64_t)table.s.tiles() * t.h_kv;
        mine_heads += table.s.nq > 0 ? t.h_kv : 0;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)lane >= o) upto += x;
    }
    int64_t tiles_heads = mine_tiles << 32 | mine_heads;       // both below 2^31 in all (the entry point's limits)
#pragma unroll
    for (int o = 16; o; o /= 2) tiles_heads += __shfl_xor_sync(0xffffffffu, tiles_heads, o);
    if (lane == 31) {
        bars->warp_sum[order / 32] = upto;
        bars->warp_tiles[order / 32] = tiles_heads;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t total = 0, all_tiles = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t x = bars->warp_sum[w];
        if (w < order / 32) upto += x;
        total += x;
        all_tiles += bars->warp_tiles[w];
    }
    const bool hand_out = !PREFIX && a.counter && hand_out_tiles(total, all_tiles >> 32, all_tiles & 0xffffffff, gridDim.x, D);
    // beside the kernel for few rows, as many CTAs as this one's share of the work (prefix.cu)
    int64_t ctas = gridDim.x;
    if constexpr (PREFIX) {
        ctas = many_ctas(total, tab.plan[a.n_plan - 1].few_units, gridDim.x);
    }
    int64_t per = quot(total + ctas - 1, ctas);
    per = per > kMinUnits ? per : kMinUnits;
    const int64_t u0 = (int64_t)blockIdx.x * per;
    const int64_t u1 = u0 + per < total ? u0 + per : total;
    const bool found = !hand_out && u0 < u1 && u0 >= upto - mine && u0 < upto;
    const uint32_t who = __ballot_sync(0xffffffffu, found);
    if (who) {
        // the warp that holds the first unit finds its tile, all lanes together
        int64_t rel = u0 - (upto - mine);
        int s = s0;
        for (; found && run > 1; ++s) {              // with one sequence a thread it is at hand
            table = read_seq(tab, s, a.tpt, a.causal);
            per_head = table.s.units(table.s.tiles());
            if (rel < (int64_t)per_head * t.h_kv) break;
            rel -= (int64_t)per_head * t.h_kv;
        }
        const int src = __ffs(who) - 1;
        s = __shfl_sync(0xffffffffu, s, src);
        rel = __shfl_sync(0xffffffffu, rel, src);
        per_head = __shfl_sync(0xffffffffu, per_head, src);
        table = read_seq(tab, s, a.tpt, a.causal);
        const int head = (int)quot(rel, per_head);
        SegmentWalk w;
        w.tpt = a.tpt;
        w.causal = a.causal;
        w.snap = snap_blocks(all_tiles >> 32, gridDim.x);
        w.start(s, table, head, (int)(rel - (int64_t)head * per_head), u0, u1);
        if (lane == 0) bars->walk = w;
    }
    if (threadIdx.x == 0 && u0 >= u1) bars->walk.at = bars->walk.end = 0;
    __syncthreads();
    const uint32_t tmem = (uint32_t)uniform((int)bars->tmem_base);
    const WaitCtx wc{&bars->abort_flag, t.status, a.timeout_ns};
    const int group = a.group;
    auto two_terms = [&](const Segment& g) {
        return FINE && (g.n_tok * group <= kFineRows || (PREFIX && (g.m & kKindPrefix)));
    };

    // the join may take its place on the chip (it waits for this grid's end)
    if constexpr (!PREFIX) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true;
    if (a.inject_timeout) alive = wait_warp(wc, bar(bars->never), 0, timeout_code(kSiteInject));

    if (alive && warp == 3) {
        // ---- Scheduler: this CTA's segments, or tiles from the counter, into the jobs.
        // Tiles are taken one ahead of the rows (every reader has read the one before),
        // so that a CTA does not take what another could start on first.
        Ring<kJobs> jr, before;
        bool ok = true, more = true;
        SegmentWalk walk = bars->walk;
        // Tiles go out 32 sequences at a time, those with the most keys first (so that the
        // last ones out are short): lane l holds the group's l-th, with the group's tiles
        // up to and with its own.
        int seq0 = 0, seq32 = 0, tiles32 = 0;
        int64_t base = 0, upto32 = 0;        // the group's first tile
        auto group32 = [&](int s) {
            const SeqTable q = s + (int)lane < t.n_seq ? read_seq(t, s + (int)lane, a.tpt, a.causal) : SeqTable{};
            const int tiles = q.s.nq > 0 ? q.s.tiles() : 0;
            const int n = t.n_seq - s < 32 ? t.n_seq - s : 32;
            int rank = 0, from = (int)lane;
            for (int i = 0; i < n; ++i) {
                const int kv = __shfl_sync(0xffffffffu, q.s.kv, i);
                rank += kv > q.s.kv || (kv == q.s.kv && i < (int)lane);
            }
            for (int i = 0; i < n; ++i)
                if (__shfl_sync(0xffffffffu, rank, i) == (int)lane) from = i;
            seq32 = s + from;
            tiles32 = __shfl_sync(0xffffffffu, tiles, from);
            upto32 = (int64_t)tiles32 * t.h_kv;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto32, o);
                if ((int)lane >= o) upto32 += x;
            }
        };
        uint32_t ticket = 0;                 // lane 0's; the first while the group is read
        if (hand_out) {
            if (lane == 0) ticket = atomicAdd(a.counter, 1u);
            group32(0);
        }
        for (int n = 0; ok && more; ++n) {
            ok = wait_w(wc, bar(bars->job_empty[jr.slot]), jr.phase ^ 1, timeout_code(kSiteJobEmpty));
            if (ok && hand_out && n > 0)
                ok = wait_w(wc, bar(bars->job_empty[before.slot]), before.phase, timeout_code(kSiteJobEmpty));
            if (!ok) break;
            Segment g;
            if (hand_out) {
                if (lane == 0 && n > 0) ticket = atomicAdd(a.counter, 1u);
                const int64_t i = __shfl_sync(0xffffffffu, ticket, 0);
                more = i < (all_tiles >> 32);
                while (more && i >= base + __shfl_sync(0xffffffffu, upto32, 31)) {
                    base += __shfl_sync(0xffffffffu, upto32, 31);
                    seq0 += 32;
                    more = seq0 < t.n_seq;             // (always, of tables in order)
                    group32(seq0);
                }
                if (more) {
                    const int who32 = __ffs(__ballot_sync(0xffffffffu, i < base + upto32)) - 1;
                    const int64_t before32 = upto32 - (int64_t)tiles32 * t.h_kv;
                    const int rel = (int)(i - base - __shfl_sync(0xffffffffu, before32, who32));
                    const int n_tiles = __shfl_sync(0xffffffffu, tiles32, who32);
                    const int seq = __shfl_sync(0xffffffffu, seq32, who32);
                    const int head = rel / n_tiles;
                    // the last row tile first: under the causal mask it is the longest
                    g = whole_tile(read_seq(t, seq, a.tpt, a.causal), seq, head, n_tiles - 1 - (rel - head * n_tiles));
                }
            } else {
                more = __all_sync(0xffffffffu, walk.next(tab, g));
                if (more) g.last_cta = g.whole || !g.from_start ? 0 : (int)quot(g.tile_end - 1, per);
                if constexpr (PREFIX) {
                    // the readers know the sequence by its entries and its kind
                    if (more) {
                        const PrefixSeq v = tab.plan[g.seq];
                        g.seq = v.row;
                        g.m = v.page0 << kKindBits | v.kind;
                    }
                }
            }
            if (!more) g.j0 = g.j1 = -1;
            if (lane == 0) {
                bars->job[jr.slot] = g;
                mbar_arrive(bar(bars->job_full[jr.slot]));
            }
            __syncwarp();
            before = jr;
            jr.advance();
        }
    }
    // ---- TMA producers.  The page_table entries of a tile come 32 at a time, one a
    // lane, the next 32 on their way.  A page outside the cache reads as zeros
    // (coordinates outside the tensor map) and is reported.
    auto produce = [&](auto which, const CUtensorMap* tm, uint64_t* full, uint64_t* empty, uint32_t ring) {
        constexpr bool is_v = decltype(which)::value;
        constexpr int n_slots = is_v ? C::SV : C::SK;
        const int rows_shift = t.page_shift < 7 ? t.page_shift : 7;    // rows of a block from one page
        int slot = 0;
        uint32_t phase = 0;
        Ring<C::NQ> qr;
        int tails = 0;
        bool ok = true;
        Ring<kJobs> jr;
        Segment g;
        while (ok && next_work<PREFIX>(bars, wc, jr, g)) {
            if constexpr (!is_v) {
                // the tile's Q as soon as its buffer is free
                const int qs = qr.slot;
                ok = wait_w(wc, bar(bars->q_empty[qs]), qr.phase ^ 1, timeout_code(kSiteQEmpty));
                if (!ok) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(bars->q_full[qs]), (uint32_t)(a.tpt * group) * (D * 2));
                __syncwarp();
#pragma unroll
                for (int ch = 0; ch < P::CHUNKS; ++ch)
                    tma_load_4d_warp(sb + C::OFF_Q + qs * C::TILE + P::offset(ch), &maps.q[P::narrow(ch)], ch * 64, 0,
                                     g.head, g.q_tok, bar(bars->q_full[qs]));
                qr.advance();
            }
            const int32_t* entries = t.page_table + (int64_t)g.seq * t.max_pages + (PREFIX ? g.m >> kKindBits : 0);
            const int n_entries = (g.kv + t.page_size - 1) >> t.page_shift;
            auto entry = [&](int i) { return i < n_entries ? entries[i] : -1; };
            int window = ((g.j0 * 128) >> t.page_shift) & ~31;             // first entry of the 32 at hand
            int page_now = entry(window + (int)lane), page_next = entry(window + 32 + (int)lane);
            for (int j = g.j0; j < g.j1; ++j) {
                const int st = slot;
                const int rows = g.kv - j * 128 < 128 ? g.kv - j * 128 : 128;     // keys of the block
                const int pages = (rows + (1 << rows_shift) - 1) >> rows_shift;
                const int first = (j * 128) >> t.page_shift;                      // a block's entries share a window
                if (first >= window + 32) {
                    window += 32;
                    page_now = page_next;
                    page_next = entry(window + 32 + (int)lane);
                }
                ok = wait_w(wc, bar(empty[st]), phase ^ 1, timeout_code(is_v ? kSiteVEmpty : kSiteKEmpty));
                if (!ok) break;
                if (++slot == n_slots) {
                    slot = 0;
                    phase ^= 1;
                }
                const bool tail = is_v && rows < 128;
                const uint32_t land = bar(tail ? bars->v_tail : full[st]);
                if (lane == 0) mbar_arrive_expect_tx(land, (uint32_t)(pages << rows_shift) * (D * 2));
                __syncwarp();
#pragma unroll 2
                for (int p = 0; p < pages; ++p) {
                    const int page = __shfl_sync(0xffffffffu, page_now, first - window + p);
                    int z = page * t.h_kv + g.head;
                    if (page < 0 || page >= t.n_pages) {
                        z = -1;
                        if (lane == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
                        __syncwarp();
                    }
                    const int row = (j * 128 + (p << rows_shift)) & (t.page_size - 1);
                    const uint32_t dst = ring + st * C::TILE;
#pragma unroll
                    for (int ch = 0; ch < P::CHUNKS; ++ch)
                        tma_load_3d_warp(dst + P::offset(ch) + (uint32_t)(p << rows_shift) * P::row_bytes(ch),
                                         &tm[P::narrow(ch)], ch * 64, row, z, land);
                }
                if (tail) {
                    ok = wait_w(wc, land, tails & 1, timeout_code(kSiteVTail));
                    if (!ok) break;
                    ++tails;
                    // rows [rows, 128) of every chunk are contiguous
                    for (int ch = 0; ch < P::CHUNKS; ++ch) {
                        const uint32_t n16 = (uint32_t)(128 - rows) * (P::row_bytes(ch) / 16);
                        const uint32_t first = ring + st * C::TILE + P::offset(ch) + (uint32_t)rows * P::row_bytes(ch);
                        for (uint32_t i = lane; i < n16; i += 32) st_shared_v4(first + i * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(full[st]));
                }
            }
        }
    };
    if (alive && warp == 0) {
        produce(std::false_type{}, maps.k, bars->k_full, bars->s_full, sb + C::OFF_K);
    } else if (alive && warp == 2) {
        produce(std::true_type{}, maps.v, bars->v_full, bars->pv_done, sb + C::OFF_V);
    } else if (alive && warp == 1) {
        // ---- MMA issuer (the whole warp, see mma_ss): one stream over all blocks of
        // all segments, S of a block before P.V of the block before.  One warp issues
        // both products because the tensor pipe takes one thread's products in order:
        // S of block g + 1 may then overwrite the buffer that P.V of block g - 1 reads.
        // (Issued from two warps, with the second told that the first had issued, they
        // were seen to run out of order.)
        constexpr uint32_t IDS = idesc_bf16(128, 128, false, false);               // S = Q K^T
        constexpr uint32_t IDO = idesc_bf16(128, P::WIDE * 64, false, true);       // O += P V, wide columns
        constexpr uint32_t IDN = idesc_bf16(128, 32, false, true);                 // and the narrow chunk's
        Ring<C::SK> rs;
        Ring<C::SV> rv;
        Ring<2> bs, bv;             // score buffers of the next S and the next P.V
        Ring<C::NQ> qr;
        uint32_t o_phase = 1;       // o_free: the first tile finds O free
        bool pending = false;       // a block has its S but not its P.V
        bool first = false;         // it is its tile's first
        bool fine = false;          // its tile's P comes in two terms (kFineRows)
        auto issue_pv = [&]() -> bool {
            if (first) {
                if (!wait_w(wc, bar(bars->o_free), o_phase, timeout_code(kSiteOFree))) return false;
                o_phase ^= 1;
            }
            const uint32_t vbase = sb + C::OFF_V + rv.slot * C::TILE;
            const uint32_t tP = tmem + (bv.slot ? C::T_S1 : C::T_S0);
            const uint32_t more = first ? 0u : 1u;
            if (!wait_w(wc, bar(bars->v_full[rv.slot]), rv.phase, timeout_code(kSiteVFull))) return false;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (!wait_w(wc, bar(bars->p_full[part][bv.slot]), bv.phase, timeout_code(kSitePFull))) return false;
                tc_fence_after();
                // key slices of 16: 0, 1 | 2, 3 of half 0, and of half 1
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = 4 * (i / 2) + 2 * part + (i & 1);
                    const bool fresh = C::SPLIT ? (kk & 3) == 0 : kk == 0;         // the accumulator's first slice
                    const uint32_t tO = tmem + (C::SPLIT && kk >= 4 ? C::T_O1 : C::T_O);
                    const uint32_t tA = tP + split_a_col(kk, 128);
                    mma_ts(tO, tA, P::desc_wide(vbase, kk), IDO, fresh ? more : 1u);
                    if constexpr (P::NARROW)
                        mma_ts(tO + P::WIDE * 64, tA, P::desc_narrow(vbase, kk), IDN, fresh ? more : 1u);
                }
                if (FINE && fine) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = 4 * (i / 2) + 2 * part + (i & 1);
                        const uint32_t tO = tmem + (C::SPLIT && kk >= 4 ? C::T_O1 : C::T_O);
                        const uint32_t tA = tP + split_a_col(kk, 128) + 32;
                        mma_ts(tO, tA, P::desc_wide(vbase, kk), IDO, 1u);
                        if constexpr (P::NARROW)
                            mma_ts(tO + P::WIDE * 64, tA, P::desc_narrow(vbase, kk), IDN, 1u);
                    }
                }
            }
            mma_commit(bar(bars->pv_done[rv.slot]));
            rv.advance();
            bv.advance();
            pending = false;
            return true;
        };
        bool ok = true;
        Ring<kJobs> jr;
        Segment g;
        for (;;) {
            // At a tile boundary the previous tile's last P.V goes first unless the next
            // job is at hand (it may come only after the rows, which wait for that P.V,
            // are done with this one) ...
            if (pending && !test_wait_warp(bar(bars->job_full[jr.slot]), jr.phase)) {
                ok = issue_pv();
                if (!ok) break;
            }
            if (!next_job<true, PREFIX>(bars, wc, jr, g)) break;
            if (g.j1 <= g.j0) continue;
            // ... and its Q and first K block are resident.
            if (pending && (!test_wait_warp(bar(bars->q_full[qr.slot]), qr.phase) ||
                            !test_wait_warp(bar(bars->k_full[rs.slot]), rs.phase))) {
                ok = issue_pv();
                if (!ok) break;
            }
            ok = wait_w(wc, bar(bars->q_full[qr.slot]), qr.phase, timeout_code(kSiteQFull));
            const uint32_t qbase = sb + C::OFF_Q + qr.slot * C::TILE;
            for (int j = g.j0; j < g.j1 && ok; ++j) {
                ok = wait_w(wc, bar(bars->k_full[rs.slot]), rs.phase, timeout_code(kSiteKFull));
                if (!ok) break;
                tc_fence_after();
                const uint32_t kbase = sb + C::OFF_K + rs.slot * C::TILE;
                const uint32_t tS = tmem + (bs.slot ? C::T_S1 : C::T_S0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tS, P::desc_k(qbase, kk), P::desc_k(kbase, kk), IDS, kk > 0 ? 1u : 0u);
                mma_commit(bar(bars->s_full[rs.slot]));
                if (j == g.j1 - 1) mma_commit(bar(bars->q_empty[qr.slot]));
                rs.advance();
                bs.advance();
                if (pending) ok = issue_pv();
                pending = true;
                first = j == g.j0;
                fine = two_terms(g);
            }
            if (!ok) break;
            qr.advance();
        }
        if (ok && pending) ok = issue_pv();
        // every MMA must be complete before the CTA releases TMEM
        mma_commit(bar(bars->drain));
        wait_w(wc, bar(bars->drain), 0, timeout_code(kSiteDrain));
    } else if (alive && warp >= 4) {
        // ---- softmax / epilogue: row = TMEM lane, half = which 64 keys of a block
        const RowThread rt = row_thread();
        const int h = rt.half, r = rt.row;
        const uint32_t lane_off = rt.lane_off;
        const uint32_t tX = tmem + C::T_X + lane_off;
        float2* xch = reinterpret_cast<float2*>(smem_raw + pad + C::OFF_XCH);
        const int r_tok = r / group, r_head = r % group;       // row r: token of the tile, head of the group
        Ring<C::SK> rg;             // this block's slot of K
        Ring<C::SV> rv;             // and of V
        Ring<2> bs;                 // and its score buffer
        uint32_t tile_phase = 0, stage_phase = 0;
        bool ok = true;
        Ring<kJobs> jr;
        Segment g;
        while (ok && next_job<false, PREFIX>(bars, wc, jr, g)) {
            const int nk = g.j1 - g.j0;
            // the rows have parts in another sequence of the plan
            const bool joined = PREFIX && (g.m & kKindJoined);
            const bool live = r_tok < g.n_tok && r < a.tpt * group;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int head = g.head * group + r_head;
            const int tok = g.q_tok + (live ? r_tok : 0);
            uint16_t* orow = a.o + ((size_t)tok * t.h_q + head) * D;
            float* lrow = a.lse + (size_t)head * t.n_tokens + tok;
            if (nk == 0) {                                     // no key for any row of the tile
                if (live) {
                    for (int c = h; c < D / 8; c += 2) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (h == 0) *lrow = -INFINITY;
                    if constexpr (PREFIX) {
                        if (h == 0) a.records[record_at(t, false, tok, head)] = kRecordNone;
                    }
                }
                continue;
            }
            // keys that this row sees
            int lim = g.kv;
            if (PREFIX ? !(g.m & kKindAll) : a.causal) {
                const int seen = g.first_pos + r_tok + 1;
                lim = seen < g.kv ? (seen > 0 ? seen : 0) : g.kv;
            }
            const uint32_t tO = tmem + C::T_O + lane_off;
            const uint32_t tO1 = tmem + C::T_O1 + lane_off;
            const uint32_t tOh = (C::SPLIT && h) ? tO1 : tO;
            float m_run = -INFINITY, l_run = 0.f;
            Ring<C::SV> before = rv;                           // the block before this one
            for (int j = 0; j < nk; ++j, before = rv, rv.advance(), rg.advance(), bs.advance()) {
                const uint32_t tS = tmem + (bs.slot ? C::T_S1 : C::T_S0) + lane_off + 64 * h;
                ok = wait_warp(wc, bar(bars->s_full[rg.slot]), rg.phase, timeout_code(kSiteSFull));
                if (!ok) break;
                if (!warp_live) {                              // no row of this warp is used: only keep step
                    if constexpr (!C::SPLIT) {
                        mbar_arrive(bar(bars->xmax[bs.slot]));
                        ok = wait_warp(wc, bar(bars->xmax[bs.slot]), bs.phase, timeout_code(kSiteXmax));
                        if (!ok) break;
                    }
                    mbar_arrive(bar(bars->p_full[0][bs.slot]));
                    mbar_arrive(bar(bars->p_full[1][bs.slot]));
                    continue;
                }
                tc_fence_after();
                float x[64];
                {
                    uint32_t rr[64];
                    tmem_ld64(tS, rr);
#pragma unroll
                    for (int e = 0; e < 64; ++e) x[e] = __uint_as_float(rr[e]);
                }
                const int left = lim - ((g.j0 + j) * 128 + 64 * h);    // visible keys from this half's first on
                if (left < 64) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c >= left) x[c] = -INFINITY;
                }
                float mx4[4];                                  // four chains: one would be 32 steps long
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx4[k] = fmaxf(x[16 * k], x[16 * k + 1]);
#pragma unroll
                    for (int c = 2; c < 16; c += 2) mx4[k] = fmax3(mx4[k], x[16 * k + c], x[16 * k + c + 1]);
                }
                float mx = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]);
                if constexpr (!C::SPLIT) {
                    tmem_st1(tX + bs.slot * 2 + h, __float_as_uint(mx));
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(bar(bars->xmax[bs.slot]));
                    ok = wait_warp(wc, bar(bars->xmax[bs.slot]), bs.phase, timeout_code(kSiteXmax));
                    if (!ok) break;
                    tc_fence_after();
                    mx = fmaxf(mx, __uint_as_float(tmem_ld1(tX + bs.slot * 2 + (h ^ 1))));
                }
                const float m_new = fmaxf(m_run, mx * a.scale_log2);
                // Only rows that are used have a say: the others' queries are the next
                // tokens', or what shared memory held before, and must not decide where
                // this tile's maxima move (which its roundings follow).
                if (__any_sync(0xffffffffu, live && m_new > m_run + 8.0f)) {
                    if (j > 0) {
                        // the accumulator's last P.V (block j - 1) must be done
                        ok = wait_warp(wc, bar(bars->pv_done[before.slot]), before.phase, timeout_code(kSitePvDone));
                        if (!ok) break;
                        tc_fence_after();
                        // a row that has seen no key yet keeps its zeros
                        const float f = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new);
                        l_run *= f;
                        const uint64_t f2 = f2_pack(f, f);
                        constexpr int c_step = C::SPLIT ? 1 : 2;
#pragma unroll 1
                        for (int c32 = C::SPLIT ? 0 : h; c32 < D / 32; c32 += c_step) {
                            uint32_t rr[32];
                            tmem_ld32(tOh + c32 * 32, rr);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint64_t o2 =
                                    f2_mul(f2_pack(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1])), f2);
                                float lo, hi;
                                f2_unpack(o2, lo, hi);
                                rr[2 * e] = __float_as_uint(lo);
                                rr[2 * e + 1] = __float_as_uint(hi);
                            }
                            tmem_st32(tOh + c32 * 32, rr);
                        }
                        tmem_st_wait();
                    }
                    m_run = m_new;
                }
                // a row (or half) that has seen no key: every p is 0, not NaN
                const float m_ref = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
                const uint64_t nm2 = f2_pack(-m_ref, -m_ref);
                uint64_t acc2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                // P goes out in two parts of 32 keys a half, so that the first part's
                // products run while the second is formed.
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float lo, hi;
                        f2_unpack(f2_fma(f2_pack(x[32 * part + 2 * e], x[32 * part + 2 * e + 1]), sc2, nm2), lo, hi);
                        lo = ex2_approx(lo);
                        hi = ex2_approx(hi);
                        acc2[e & 1] = f2_add(acc2[e & 1], f2_pack(lo, hi));
                        pw[e] = pack_bf16x2(lo, hi);
                    }
                    tmem_st16(tS + 16 * part, pw);
                    if (two_terms(g)) {
                        // what the rounding left, into the half's other 32 columns (p formed
                        // again, which costs the other tiles no registers)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float lo, hi;
                            f2_unpack(f2_fma(f2_pack(x[32 * part + 2 * e], x[32 * part + 2 * e + 1]), sc2, nm2), lo, hi);
                            pw[e] = pack_bf16x2(ex2_approx(lo) - __uint_as_float(pw[e] << 16),
                                                ex2_approx(hi) - __uint_as_float(pw[e] & 0xffff0000u));
                        }
                        tmem_st16(tS + 32 + 16 * part, pw);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(bar(bars->p_full[part][bs.slot]));
                }
                {
                    float lo, hi;
                    f2_unpack(f2_add(acc2[0], acc2[1]), lo, hi);
                    l_run += lo + hi;
                }
            }
            if (!ok) break;
            // Final row statistics: O = a0 O_0 + a1 O_1 (SPLIT), O = a0 O (else); a
            // row that saw no key has l = 0 and gets zeros.  (Compared with 0: the sum of
            // a row that saw a NaN score is NaN, and has to reach O and the LSE.)
            float a0 = 0.f, a1 = 0.f, lse2 = -INFINITY;
            // a full tile's O leaves through the stage: free once its last store has read it
            const bool staged = C::STAGE_O && g.whole && g.n_tok == a.tpt;
            if (staged && h == 0 && r == 0) bulk_wait_read0();
            if constexpr (C::SPLIT) {
                if (h == 1) xch[r] = make_float2(m_run, l_run);
                mbar_arrive(bar(bars->lsum));
                ok = wait_warp(wc, bar(bars->lsum), tile_phase, timeout_code(kSiteLsum));
                if (!ok) break;
                if (h == 0) {
                    const float2 o1 = xch[r];
                    const float m = fmaxf(m_run, o1.x);
                    const float m_ref = (m == -INFINITY) ? 0.f : m;
                    const float f0 = ex2_approx(m_run - m_ref), f1 = ex2_approx(o1.x - m_ref);
                    const float l_tot = l_run * f0 + o1.y * f1;
                    const float inv = l_tot == 0.f ? 0.f : 1.0f / l_tot;
                    a0 = f0 * inv;
                    a1 = f1 * inv;
                    lse2 = l_tot == 0.f ? -INFINITY : m_ref + log2f(l_tot);
                    xch[r] = make_float2(a0, a1);
                }
                mbar_arrive(bar(bars->lsum2));
                ok = wait_warp(wc, bar(bars->lsum2), tile_phase, timeout_code(kSiteLsum));
                if (!ok) break;
                if (h == 1) {
                    const float2 f = xch[r];
                    a0 = f.x;
                    a1 = f.y;
                }
            } else {
                tmem_st1(tX + 4 + h, __float_as_uint(l_run));
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(bars->lsum));
                ok = wait_warp(wc, bar(bars->lsum), tile_phase, timeout_code(kSiteLsum));
                if (!ok) break;
                tc_fence_after();
                const float l_tot = l_run + __uint_as_float(tmem_ld1(tX + 4 + (h ^ 1)));
                a0 = l_tot == 0.f ? 0.f : 1.0f / l_tot;
                lse2 = l_tot == 0.f ? -INFINITY : m_run + log2f(l_tot);
            }
            ok = wait_warp(wc, bar(bars->pv_done[before.slot]), before.phase, timeout_code(kSitePvDone));
            if (!ok) break;
            tc_fence_after();
            if (warp_live) {
                // a finished row goes to O; others, as fp32, to the workspace
                const bool done = g.whole && !joined;
                size_t prow = part_row(blockIdx.x, g.from_start ? 1 : 0) + r;
                if (PREFIX && g.whole) prow = whole_row(t, g.m & kKindPrefix, tok, head);
                float* part = reinterpret_cast<float*>(a.ws) + prow * D;
                if (live && h == 0) {
                    if (done)
                        *lrow = lse2 * 0.693147180559945309f;
                    else
                        reinterpret_cast<float*>(a.ws + (PREFIX ? a.lse_offset : ws_lse_offset(D)))[prow] = lse2;
                    if constexpr (PREFIX) {
                        if (g.from_start)
                            a.records[record_at(t, g.m & kKindPrefix, tok, head)] =
                                done ? kRecordNone : make_record(g.whole, joined, blockIdx.x, g.last_cta, r);
                    }
                }
                // batches of shared pages: the rows that this lane stores a piece of, 8 rows apart
                size_t turned[4] = {};
                uint32_t turned_live = 0;
                if constexpr (PREFIX) {
                    if (!done) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r2 = (r & ~31) + (int)lane / 4 + 8 * i, t2 = r2 / group;
                            turned[i] = g.whole ? whole_row(t, g.m & kKindPrefix, g.q_tok + t2, g.head * group + r2 - t2 * group)
                                                : part_row(blockIdx.x, g.from_start ? 1 : 0) + r2;
                            if (t2 < g.n_tok && r2 < a.tpt * group) turned_live |= 1u << i;
                        }
                    }
                }
                // The TMEM loads are warp-collective; only the stores are guarded.
#pragma unroll 1
                for (int c32 = h; c32 < D / 32; c32 += 2) {
                    uint32_t rr[32];
                    tmem_ld32(tO + c32 * 32, rr);
                    float f[32];
                    if constexpr (C::SPLIT) {
                        uint32_t r1[32];
                        tmem_ld32(tO1 + c32 * 32, r1);
                        // a half without a visible key has an accumulator of zeros (p = 0)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            f[e] = __uint_as_float(rr[e]) * a0 + __uint_as_float(r1[e]) * a1;
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(rr[e]) * a0;
                    }
                    if (done) {
#pragma unroll
                        for (int u4 = 0; u4 < 4; ++u4) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(f[8 * u4 + 2 * e], f[8 * u4 + 2 * e + 1]);
                            if (staged)
                                st_shared_v4(sb + C::OFF_OST + G::template unit_offset<128>(r, c32 * 32 + 8 * u4), w[0],
                                             w[1], w[2], w[3]);
                            else if (live)
                                reinterpret_cast<uint4*>(orow)[c32 * 4 + u4] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if constexpr (PREFIX) {
                        // 16 columns of 32 rows at a time, so that the stores are of whole sectors
                        // (a thread storing its own row cost 2 us a tile)
                        const uint32_t turn = sb + C::OFF_TURN + (warp - 4) * 2048;
#pragma unroll
                        for (int c16 = 0; c16 < 2; ++c16) {
                            __syncwarp();
#pragma unroll
                            for (int u4 = 0; u4 < 4; ++u4)
                                st_shared_v4(turn + lane * 64 + ((u4 ^ (lane >> 1 & 3)) * 16),
                                             __float_as_uint(f[16 * c16 + 4 * u4]), __float_as_uint(f[16 * c16 + 4 * u4 + 1]),
                                             __float_as_uint(f[16 * c16 + 4 * u4 + 2]), __float_as_uint(f[16 * c16 + 4 * u4 + 3]));
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t r2 = lane / 4 + 8 * i;
                                const uint4 x = ld_shared_v4(turn + r2 * 64 + (((lane & 3) ^ (r2 >> 1 & 3)) * 16));
                                if (turned_live >> i & 1)
                                    reinterpret_cast<uint4*>(reinterpret_cast<float*>(a.ws) + turned[i] * D + c32 * 32 +
                                                             16 * c16)[lane & 3] = x;
                            }
                        }
                    } else if (live) {
#pragma unroll
                        for (int u4 = 0; u4 < 8; ++u4)
                            reinterpret_cast<float4*>(part)[c32 * 8 + u4] =
                                make_float4(f[4 * u4], f[4 * u4 + 1], f[4 * u4 + 2], f[4 * u4 + 3]);
                    }
                }
                if (!PREFIX && !g.whole && g.from_start && h == 0 && r == 0) {
                    CutTile* cut = reinterpret_cast<CutTile*>(a.ws + ws_cut_offset(D)) + blockIdx.x;
                    cut->q_tok = g.q_tok;
                    cut->n_rows = g.n_tok * group;
                    cut->head = g.head;
                    cut->last_cta = g.last_cta;
                }
            }
            tc_fence_before();
            mbar_arrive(bar(bars->o_free));
            tile_phase ^= 1;
            if (staged) {
                fence_proxy_async_smem();
                mbar_arrive(bar(bars->ost_full));
                if (warp == 4) {
                    ok = wait_warp(wc, bar(bars->ost_full), stage_phase, timeout_code(kSiteStage));
                    if (!ok) break;
                    if (lane == 0) {
                        for (int ch = 0; ch < G::NCH; ++ch)
                            tma_store_4d(&maps.o, sb + C::OFF_OST + ch * C::CHUNK, ch * G::CW, 0, g.head, g.q_tok);
                        bulk_commit();
                    }
                    __syncwarp();
                }
                stage_phase ^= 1;
            }
        }
        // the last O store must have read the stage before the CTA exits
        if (h == 0 && r == 0) bulk_wait_read0();
    }

    __syncthreads();
    if (bars->abort_flag) {
        // Let any copy or MMA issued before the abort land before TMEM and
        // shared memory are released.
        for (int k = 0; k < 20; ++k) __nanosleep(50000);
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace ac
