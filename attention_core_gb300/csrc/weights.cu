// weights.cu -- the attention weight that each key of a paged cache gathers, on sm_103a:
//
//     a'_j = (j older than the call's tokens ? decay a_j : 0)
//            + sum over new tokens t that see j, heads h of the group: exp(scale q_th . k_j - LSE_th)
//
// per (sequence, KV head, key), with the LSE that the attention over the same cache
// returned.  Scores are formed the other way round, S^T = K Q^T with the keys as the 128
// TMEM lanes: a thread owns a key and adds up its columns, so the sum over rows needs no
// exchange between threads, and each weight has one owner and one order of addition.
//
// Bounds: single tokens the keys' bytes; chunks the products (1024 cycles for a row tile
// and 256 keys at d = 128) and the exponentials (1024: 4 cycles for a warp's), beside which
// the issuing and summing warps' own work still stands.  Measured on one GB300:
//   one new token of 64 sequences of up to 8192 keys, 64/8 heads of 128   114 us (6.0 TB/s)
//   2048 new tokens over 8192 keys, 64/8 heads of 128            186 us (1.30 PFLOP/s)
//   8 sequences, up to 500 new tokens over 4001 keys, 16 heads of 160          43 us
//   one new token over 500 keys                                     9 us in a graph
// Tried and left out: row tiles of 256 rows whose columns a half's two warpgroups share (half
// the products and commits, one score buffer a half: 203 us); a part of the exponentials by a
// polynomial on the FMA pipe (they do not bound the loop: 190 -> 236 us); two issuing warps,
// one for each half (192 us, and one launch in about 600 of single tokens ended in a launch
// failure; with one issuing warp 24000 launches gave the same bits).  That form's source is
// not kept.  What a second issuer changes, by reading: a row tile's slot is free after two
// commits, not one; and a commit covers the products of its own thread alone, so each issuer
// needs a drain barrier of its own.  With one between them the faster issuer's commit lets
// both leave, and the other's last commits can arrive when the CTA's shared memory is no
// longer its own: rare, with right results before, as was seen.  Here one thread issues and
// commits everything, waits for its last commit before the CTA's last barrier, and TMEM is
// given back behind that one.
//
// Persistent, one CTA per SM, equal shares of the work (weights_sched.cuh).  640 threads:
//   warp 0  runs of items, in a ring of jobs that the others read, and their K by TMA: an
//           item's 256 keys as two tiles of 128
//   warp 2  row tiles: Q by TMA, and the rows' -LSE log2 e with a bit per row that counts
//           (of a token of the sequence, its LSE not -inf).  A sequence of one tile keeps
//           it for the whole run.
//   warp 1  issues the tcgen05 MMAs: per row tile and half of the item one [128 keys x
//           rows] product, N only as wide as the tile has rows
//   warps 4-19  exponentials and sums: two warpgroups for each half, which take its row
//           tiles in turn, each with a TMEM buffer of its own
// A score is fp32; a tile's exponentials are summed in four fp32 chains, and the tiles'
// sums on top, so that thousands of rows lose no more than their tiles' count.
#include <stddef.h>

#include "paged_attn.cuh"
#include "weights_sched.cuh"

namespace ac {

namespace {

constexpr int kSumWarps = 16;                       // four warpgroups, from warp 4 on
constexpr int kWeightsThreads = 32 * (4 + kSumWarps);

// Batches of single tokens: row tiles of 32 rows, and the shared memory for K.
constexpr int kFewWeightRows = 32;

template <int D, int ROWS>
struct WeightsCfg {
    static constexpr bool FEW = ROWS < 128;
    static constexpr uint32_t TILE = PagedGeom<D>::TILE, QTILE = PagedGeom<D, ROWS>::TILE;
    static constexpr int SK = FEW ? (D <= 96 ? 8 : D <= 128 ? 6 : 5) : (D <= 64 ? 8 : D <= 96 ? 5 : 3);   // K tiles
    static constexpr int SQ = FEW ? 2 : D <= 96 ? 4 : D <= 128 ? 3 : 2;                                   // row tiles
    static constexpr uint32_t OFF_Q = SK * TILE;
    static constexpr uint32_t OFF_BAR = OFF_Q + SQ * QTILE;
    static constexpr uint32_t BAR_BYTES = 6144;
    static constexpr uint32_t SMEM = OFF_BAR + BAR_BYTES + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

struct WeightsBars {
    float nlse[4][128];             // a row tile's -LSE log2 e
    uint32_t counts[4][4];          // its rows that count
    float xch[2][2][128];
    uint64_t k_full[8], k_empty[8];
    uint64_t q_full[4], l_full[4];
    uint64_t s_full[2][2];          // [half][warpgroup]
    uint64_t job_full[kJobs];
    uint64_t drain, never;
    uint64_t q_empty[4];
    uint64_t s_empty[2][2];         // the warps of one warpgroup
    uint64_t x_full[2][2], x_empty[2][2];   // [half][buffer]: sums of a half's second warpgroup
    uint64_t l_empty[4];            // all summing warps
    uint64_t job_empty[kJobs];
    int64_t warp_sum[kWeightsThreads / 32];
    ItemWalk walk;
    uint32_t tmem_base;
    int32_t abort_flag;
    ItemRun job[kJobs];
};
static_assert(sizeof(WeightsBars) <= WeightsCfg<64, 128>::BAR_BYTES, "barrier block");
constexpr int kWeightsReaders = 2 + kSumWarps;

enum : int32_t {
    kSiteWInject = 32, kSiteWJobEmpty, kSiteWJobFull, kSiteWKEmpty, kSiteWKFull, kSiteWQEmpty, kSiteWQFull,
    kSiteWLEmpty, kSiteWLFull, kSiteWSEmpty, kSiteWSFull, kSiteWXEmpty, kSiteWXFull, kSiteWDrain
};

// A cut item, written by the CTA that has its first piece (slot 1 of its own two; the
// later pieces are in slot 0 of the CTAs after it).
struct CutItem {
    int32_t last_cta;    // 0: this CTA cut no item at its end
    int32_t seq, head, item, old, kv;
    int32_t pad[2];
};
constexpr size_t kWeightsParts = (size_t)kPagedMaxCtas * 2 * kItemKeys * sizeof(float);

__device__ __forceinline__ uint64_t ex2_pair(uint64_t x)
{
    float lo, hi;
    f2_unpack(x, lo, hi);
    return f2_pack(ex2_approx(lo), ex2_approx(hi));
}

__device__ __forceinline__ bool next_run(WeightsBars* bars, const WaitCtx& wc, Ring<kJobs>& jr, ItemRun& g)
{
    if (!wait_w(wc, smem_u32(&bars->job_full[jr.slot]), jr.phase, timeout_code(kSiteWJobFull))) return false;
    const ItemRun& s = bars->job[jr.slot];
    g.seq = uniform(s.seq);
    g.head = uniform(s.head);
    g.q0 = uniform(s.q0);
    g.nq = uniform(s.nq);
    g.kv = uniform(s.kv);
    g.i0 = uniform(s.i0);
    g.i1 = uniform(s.i1);
    g.whole = uniform(s.whole);
    g.m0 = uniform(s.m0);
    g.m1 = uniform(s.m1);
    g.from_start = uniform(s.from_start);
    g.last_cta = uniform(s.last_cta);
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(smem_u32(&bars->job_empty[jr.slot]));
    jr.advance();
    return g.i0 >= 0;
}

}  // namespace

// PADDED: row tiles of 128 with rows that no tile has, whose scores of infinite keys are
// looked for: 3% of a chunk's time, which batches of full tiles go without.
template <int D, int ROWS, bool PADDED>
__global__ void __launch_bounds__(kWeightsThreads, 1)
paged_weights_kernel(const __grid_constant__ PagedMaps maps, const WeightsArgs a)
{
    using P = PagedGeom<D>;
    using PQ = PagedGeom<D, ROWS>;
    using C = WeightsCfg<D, ROWS>;
    const PagedTables& t = a.t;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    const uint32_t sb = raw + pad;
    WeightsBars* bars = reinterpret_cast<WeightsBars*>(smem_raw + pad + C::OFF_BAR);
    auto bar = [](uint64_t& b) { return smem_u32(&b); };
    const uint32_t warp = (uint32_t)uniform((int)warp_id()), lane = lane_id();
    CutItem* cuts = reinterpret_cast<CutItem*>(a.ws + kWeightsParts);
    float* parts = reinterpret_cast<float*>(a.ws) + (size_t)blockIdx.x * 2 * kItemKeys;

    if (warp == 3) {
        uint64_t* first = bars->k_full;
        const int once = (int)(&bars->s_empty[0][0] - first), four = (int)(bars->l_empty - &bars->s_empty[0][0]);
        for (int i = lane; i < once; i += 32) mbar_init(bar(first[i]), 1);
        if ((int)lane < four) mbar_init(bar((&bars->s_empty[0][0])[lane]), 4);
        if (lane < 4) mbar_init(bar(bars->l_empty[lane]), kSumWarps);
        if (lane < kJobs) mbar_init(bar(bars->job_empty[lane]), kWeightsReaders);
        if (lane == 0) {
            bars->abort_flag = 0;
            cuts[blockIdx.x].last_cta = 0;
        }
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < (P::NARROW ? 2 : 1); ++i) {
            tma_prefetch_desc(&maps.q[i]);
            tma_prefetch_desc(&maps.k[i]);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    // Rows that no tile has (head groups that do not divide the tile): zeros, so that their
    // scores of finite keys are finite and -inf takes their place in the exponent.
    const int tile_rows = a.tpt * a.group;
    if (tile_rows < ROWS) {
        for (int s = 0; s < C::SQ; ++s)
            for (int ch = 0; ch < PQ::CHUNKS; ++ch) {
                const uint32_t first = sb + C::OFF_Q + s * C::QTILE + PQ::offset(ch) + tile_rows * PQ::row_bytes(ch);
                const uint32_t n16 = (uint32_t)(ROWS - tile_rows) * (PQ::row_bytes(ch) / 16);
                for (uint32_t i = threadIdx.x; i < n16; i += kWeightsThreads) st_shared_v4(first + i * 16, 0u, 0u, 0u, 0u);
            }
        fence_proxy_async_smem();
    }

    // this CTA's share, as in paged_attn.cuh
    const int order = ((int)threadIdx.x + kWeightsThreads - 128) % kWeightsThreads;     // warp 4 first
    const int run = (t.n_seq + kWeightsThreads - 1) / kWeightsThreads;
    const int s0 = order * run < t.n_seq ? order * run : t.n_seq;
    const int s1 = s0 + run < t.n_seq ? s0 + run : t.n_seq;
    int64_t mine = 0;
    int per_head = 0;
    SeqTable table{};
    for (int s = s0; s < s1; ++s) {
        table = read_seq(t, s, a.tpt, a.causal);
        if (table.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
        const ItemShape sh = item_shape(table);
        per_head = sh.units(sh.items());
        mine += (int64_t)per_head * t.h_kv;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)lane >= o) upto += x;
    }
    if (lane == 31) bars->warp_sum[order / 32] = upto;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWeightsThreads / 32; ++w) {
        const int64_t x = bars->warp_sum[w];
        if (w < order / 32) upto += x;
        total += x;
    }
    int64_t per = quot(total + gridDim.x - 1, gridDim.x);
    per = per > 1 ? per : 1;
    const int64_t u0 = (int64_t)blockIdx.x * per;
    const int64_t u1 = u0 + per < total ? u0 + per : total;
    const uint32_t who = __ballot_sync(0xffffffffu, u0 < u1 && u0 >= upto - mine && u0 < upto);
    if (who) {
        int64_t rel = u0 - (upto - mine);
        int s = s0;
        if ((who >> lane) & 1) {
            for (;; ++s) {
                table = read_seq(t, s, a.tpt, a.causal);
                const ItemShape sh = item_shape(table);
                per_head = sh.units(sh.items());
                if (rel < (int64_t)per_head * t.h_kv) break;
                rel -= (int64_t)per_head * t.h_kv;
            }
        }
        const int src = __ffs(who) - 1;
        s = __shfl_sync(0xffffffffu, s, src);
        rel = __shfl_sync(0xffffffffu, rel, src);
        per_head = __shfl_sync(0xffffffffu, per_head, src);
        table = read_seq(t, s, a.tpt, a.causal);
        const int head = (int)quot(rel, per_head);
        ItemWalk w;
        w.tpt = a.tpt;
        w.causal = a.causal;
        w.per = per;
        w.start(s, table, head, (int)(rel - (int64_t)head * per_head), u0, u1);
        if (lane == 0) bars->walk = w;
    }
    if (threadIdx.x == 0 && u0 >= u1) bars->walk.at = bars->walk.end = 0;
    __syncthreads();
    const uint32_t tmem = (uint32_t)uniform((int)bars->tmem_base);
    const WaitCtx wc{&bars->abort_flag, t.status, a.timeout_ns};
    const int group = a.group, tpt = a.tpt;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true;
    if (a.inject_timeout) alive = wait_warp(wc, bar(bars->never), 0, timeout_code(kSiteWInject));

    // The row tiles of item i in a run: all from the first that sees its first key, or the piece's.
    auto shape = [&](const ItemRun& g) { return ItemShape{g.nq, g.kv, tpt, a.causal}; };

    if (alive && warp == 0) {
        // ---- runs of items for everyone, and their K: page_table entries 32 at a time, one a
        // lane, the next 32 on their way.  A page outside the cache reads as zeros and is
        // reported.
        const int rows_shift = t.page_shift < 7 ? t.page_shift : 7;
        Ring<C::SK> rk;
        Ring<kJobs> jr;
        ItemWalk walk = bars->walk;
        ItemRun g{};
        bool ok = true;
        for (;;) {
            ok = wait_w(wc, bar(bars->job_empty[jr.slot]), jr.phase ^ 1, timeout_code(kSiteWJobEmpty));
            if (!ok) break;
            const bool more = __all_sync(0xffffffffu, walk.next(t, g));
            if (!more) g.i0 = -1;
            if (lane == 0) {
                bars->job[jr.slot] = g;
                mbar_arrive(bar(bars->job_full[jr.slot]));
            }
            __syncwarp();
            jr.advance();
            if (!more) break;
            g.seq = uniform(g.seq);
            g.head = uniform(g.head);
            g.kv = uniform(g.kv);
            g.i0 = uniform(g.i0);
            g.i1 = uniform(g.i1);
            const int32_t* entries = t.page_table + (int64_t)g.seq * t.max_pages;
            const int n_entries = (g.kv + t.page_size - 1) >> t.page_shift;
            auto entry = [&](int i) { return i < n_entries ? entries[i] : -1; };
            int window = ((g.i0 * kItemKeys) >> t.page_shift) & ~31;
            int page_now = entry(window + (int)lane), page_next = entry(window + 32 + (int)lane);
            for (int j = 2 * g.i0; ok && j < 2 * g.i1 && j * 128 < g.kv; ++j) {
                const int rows = g.kv - j * 128 < 128 ? g.kv - j * 128 : 128;
                const int pages = (rows + (1 << rows_shift) - 1) >> rows_shift;
                const int first = (j * 128) >> t.page_shift;
                if (first >= window + 32) {
                    window += 32;
                    page_now = page_next;
                    page_next = entry(window + 32 + (int)lane);
                }
                ok = wait_w(wc, bar(bars->k_empty[rk.slot]), rk.phase ^ 1, timeout_code(kSiteWKEmpty));
                if (!ok) break;
                const uint32_t land = bar(bars->k_full[rk.slot]);
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
                    const uint32_t dst = sb + rk.slot * C::TILE;
#pragma unroll
                    for (int ch = 0; ch < P::CHUNKS; ++ch)
                        tma_load_3d_warp(dst + P::offset(ch) + (uint32_t)(p << rows_shift) * P::row_bytes(ch),
                                         &maps.k[P::narrow(ch)], ch * 64, row, z, land);
                }
                rk.advance();
            }
            if (!ok) break;
        }
    } else if (alive && warp == 2) {
        // ---- row tiles
        constexpr int W = ROWS / 32;
        int r_tok[W], r_head[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            r_tok[k] = (int)(lane + 32 * k) / group;
            r_head[k] = (int)(lane + 32 * k) - r_tok[k] * group;
        }
        Ring<C::SQ> rq;
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        // a tile's LSEs are on their way while the tile before it is placed
        float l_next[W];
        auto fetch = [&](int m) {
            const int tok0 = g.q0 + m * tpt;
            const int n_tok = g.nq - m * tpt < tpt ? g.nq - m * tpt : tpt;
#pragma unroll
            for (int k = 0; k < W; ++k)
                l_next[k] = r_tok[k] < n_tok
                                ? a.lse[(size_t)(g.head * group + r_head[k]) * t.n_tokens + tok0 + r_tok[k]]
                                : -INFINITY;
        };
        auto load = [&](int m, int next) -> bool {
            const int tok0 = g.q0 + m * tpt;
            float l[W];
#pragma unroll
            for (int k = 0; k < W; ++k) l[k] = l_next[k];
            if (next >= 0) fetch(next);
            if (!wait_w(wc, bar(bars->q_empty[rq.slot]), rq.phase ^ 1, timeout_code(kSiteWQEmpty))) return false;
            if (lane == 0) mbar_arrive_expect_tx(bar(bars->q_full[rq.slot]), (uint32_t)(tpt * group) * (D * 2));
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < P::CHUNKS; ++ch)
                tma_load_4d_warp(sb + C::OFF_Q + rq.slot * C::QTILE + PQ::offset(ch), &maps.q[P::narrow(ch)], ch * 64,
                                 0, g.head, tok0, bar(bars->q_full[rq.slot]));
            if (!wait_w(wc, bar(bars->l_empty[rq.slot]), rq.phase ^ 1, timeout_code(kSiteWLEmpty))) return false;
            // a row that no tile has counts, and adds exp(-inf)
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const bool none = (int)lane + 32 * k >= tpt * group, counts = none || l[k] != -INFINITY;
                const uint32_t bits = __ballot_sync(0xffffffffu, counts);
                if (lane == 0) bars->counts[rq.slot][k] = bits;
                bars->nlse[rq.slot][lane + 32 * k] =
                    none ? -INFINITY : counts ? l[k] * -1.44269504088896340736f : 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bars->l_full[rq.slot]));
            rq.advance();
            return true;
        };
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles();
            int m = g.whole ? s.first_tile(g.i0 * kItemKeys) : g.m0;
            fetch(m);
            if (tiles == 1) {
                ok = load(0, -1);
                continue;
            }
            const int m1 = g.whole ? tiles : g.m1;
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const int after = i + 1 < g.i1 ? s.first_tile((i + 1) * kItemKeys) : -1;
                for (; ok && m < m1; ++m) ok = load(m, m + 1 < m1 ? m + 1 : after);
                m = after;
            }
        }
    } else if (alive && warp == 1) {
        // ---- MMA issuer: S^T of both halves for the tiles whose rows see them, for each
        // half's two warpgroups in turn
        Ring<C::SK> rk;
        Ring<C::SQ> rq;
        int turn = 0;               // the tile's warpgroups
        uint32_t s_phase = 0xf;     // bit 2 half + turn: parity of the buffer's next release
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        auto product = [&](uint32_t tS, uint32_t kbase, uint32_t qbase, uint32_t ids) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tS, P::desc_k(kbase, kk), PQ::desc_k(qbase, kk), ids, kk > 0 ? 1u : 0u);
        };
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles(), m1 = g.whole ? tiles : g.m1;
            const int last_rows = (g.nq - (tiles - 1) * tpt) * group;
            // all of a full tile's columns, those of rows that no tile has among them: they are read
            const uint32_t ids_all = idesc_bf16(128, ROWS, false, false);
            const uint32_t ids_last =
                last_rows == tpt * group
                    ? ids_all : idesc_bf16(128, 0, false, false) | (uint32_t)((last_rows + 15) / 16 * 2) << 17;
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const bool two = g.kv - i * kItemKeys > 128;
                const int first = g.whole ? s.first_tile(i * kItemKeys) : g.m0;
                int from2 = two ? s.first_tile(i * kItemKeys + 128) : m1;
                if (from2 < first) from2 = first;
                Ring<C::SK> rk2 = rk;
                if (two) rk2.advance();
                const uint32_t kbase = sb + rk.slot * C::TILE, kbase2 = sb + rk2.slot * C::TILE;
                ok = wait_w(wc, bar(bars->k_full[rk.slot]), rk.phase, timeout_code(kSiteWKFull));
                for (int m = first; ok && m < m1; ++m) {
                    const bool both = m >= from2;
                    const uint32_t q_bar = bar(bars->q_full[rq.slot]), s0_bar = bar(bars->s_empty[0][turn]),
                                   s1_bar = bar(bars->s_empty[1][turn]);
                    const uint32_t s0_phase = s_phase >> turn & 1, s1_phase = s_phase >> (2 + turn) & 1;
                    // one look at all three; each is waited for only where one is not there
                    bool seen = mbar_test_wait(q_bar, rq.phase);
                    seen &= mbar_test_wait(s0_bar, s0_phase);
                    seen &= !both || mbar_test_wait(s1_bar, s1_phase);
                    const bool ready = __all_sync(0xffffffffu, seen);
                    if (!ready) {
                        ok = wait_w(wc, q_bar, rq.phase, timeout_code(kSiteWQFull)) &&
                             wait_w(wc, s0_bar, s0_phase, timeout_code(kSiteWSEmpty));
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint32_t qbase = sb + C::OFF_Q + rq.slot * C::QTILE;
                    const uint32_t ids = m == tiles - 1 ? ids_last : ids_all;
                    product(tmem + (uint32_t)turn * 128, kbase, qbase, ids);
                    mma_commit(bar(bars->s_full[0][turn]));
                    s_phase ^= 1u << turn;
                    if (m == m1 - 1) mma_commit(bar(bars->k_empty[rk.slot]));
                    if (both) {
                        if (m == from2) ok = wait_w(wc, bar(bars->k_full[rk2.slot]), rk2.phase, timeout_code(kSiteWKFull));
                        ok = ok && (ready || wait_w(wc, s1_bar, s1_phase, timeout_code(kSiteWSEmpty)));
                        if (!ok) break;
                        tc_fence_after();
                        product(tmem + 256 + (uint32_t)turn * 128, kbase2, qbase, ids);
                        mma_commit(bar(bars->s_full[1][turn]));
                        s_phase ^= 4u << turn;
                        if (m == m1 - 1) mma_commit(bar(bars->k_empty[rk2.slot]));
                    }
                    turn ^= 1;
                    if (tiles > 1 || i == g.i1 - 1) {
                        mma_commit(bar(bars->q_empty[rq.slot]));
                        rq.advance();
                    }
                }
                if (!ok) break;
                // a second half that no tile of a piece sees has to land before its slot is free
                if (two && from2 >= m1) {
                    ok = wait_w(wc, bar(bars->k_full[rk2.slot]), rk2.phase, timeout_code(kSiteWKFull));
                    if (!ok) break;
                    mma_commit(bar(bars->k_empty[rk2.slot]));
                }
                rk = rk2;
                rk.advance();
            }
        }
        mma_commit(bar(bars->drain));
        wait_w(wc, bar(bars->drain), 0, timeout_code(kSiteWDrain));
    } else if (alive && warp >= 4) {
        // ---- sums: a thread per key of its half, the half's tiles in turn for its two
        // warpgroups, u; the second's sum goes to the first, where an item has several tiles
        const int w = (int)(warp - 4) / 8, u = (int)(warp - 4) / 4 & 1;
        const int row = (int)(warp & 3) * 32 + (int)lane;
        const uint32_t lane_off = (warp & 3u) * 32u << 16;
        const uint32_t tS = tmem + (uint32_t)(w * 2 + u) * 128 + lane_off;
        float (*xch)[128] = bars->xch[w];
        Ring<C::SQ> rq;
        Ring<2> rx;
        uint32_t s_phase = 0;
        int turn = 0;               // whose the next tile is
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
        const size_t length = (size_t)t.max_pages * t.page_size;
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles(), e = g.kv - g.nq, m1 = g.whole ? tiles : g.m1;
            const size_t line = ((size_t)g.seq * t.h_kv + g.head) * length;
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const int key0 = i * kItemKeys + w * 128, key = key0 + row;
                const int first = g.whole ? s.first_tile(i * kItemKeys) : g.m0;
                const int from = key0 < g.kv ? s.first_tile(key0) : m1;
                const bool sole = tiles == 1, owner = sole ? turn == u && key0 < g.kv : u == 0;
                float old = 0.f, sum = 0.f;
                if (owner && g.whole && key < e) old = a.in[line + key];
                for (int m = first; m < m1; ++m) {
                    if (tiles > 1 || i == g.i0) {
                        ok = wait_warp(wc, bar(bars->l_full[rq.slot]), rq.phase, timeout_code(kSiteWLFull));
                        if (!ok) break;
                    }
                    if (turn == u) {
                        if (m >= from) {
                            ok = wait_warp(wc, bar(bars->s_full[w][u]), s_phase, timeout_code(kSiteWSFull));
                            if (!ok) break;
                            s_phase ^= 1;
                            tc_fence_after();
                            const float* nl = bars->nlse[rq.slot];
                            const uint4 counts = *reinterpret_cast<const uint4*>(bars->counts[rq.slot]);
                            const int pos = e + m * tpt;                        // of the tile's first token
                            const bool plain = !C::FEW && (counts.x & counts.y & counts.z & counts.w) == 0xffffffffu &&
                                               (!a.causal || key0 + 127 <= pos);
                            float part = 0.f;
                            if (plain) {
                                uint64_t acc[4] = {0, 0, 0, 0};
                                uint32_t x[2][32];       // the next 32 columns are on their way
                                tmem_ld32_issue(tS, x[0]);
#pragma unroll
                                for (int c0 = 0; c0 < 128; c0 += 32) {
                                    uint32_t (&y)[32] = x[c0 / 32 & 1];
                                    tmem_ld_wait(y);
                                    if (c0 < 96) tmem_ld32_issue(tS + c0 + 32, x[c0 / 32 + 1 & 1]);
#pragma unroll
                                    for (int c = 0; c < 32; c += 4) {
                                        const float4 n4 = *reinterpret_cast<const float4*>(nl + c0 + c);
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            const int pair = c / 2 + h;
                                            const uint64_t z = f2_fma(f2_pack(__uint_as_float(y[2 * pair]),
                                                                              __uint_as_float(y[2 * pair + 1])),
                                                                      sc2, h ? f2_pack(n4.z, n4.w) : f2_pack(n4.x, n4.y));
                                            acc[pair & 3] =
                                                f2_add(acc[pair & 3], ex2_pair(z));
                                        }
                                    }
                                }
                                float lo, hi;
                                f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
                                part = lo + hi;
                            }
                            // an infinite key's score is NaN in the rows that no tile has (0 x inf): it is
                            // summed again, without them
                            const bool again = plain && part != part;
                            if (!plain || (PADDED && __any_sync(0xffffffffu, again))) {
                                // rows that do not count, or whose mask hides this key, are left out
                                // whatever their score is
                                const int rows = (g.nq - m * tpt < tpt ? g.nq - m * tpt : tpt) * group;
                                const int skip0 = a.causal && key > pos ? (key - pos) * group : 0;
                                float counted = 0.f;
#pragma unroll 1
                                for (int c0 = 0; c0 < rows; c0 += 32) {
                                    uint32_t x[32];
                                    tmem_ld32(tS + c0, x);
                                    uint32_t bits = bars->counts[rq.slot][c0 / 32];
                                    if (rows - c0 < 32) bits &= (1u << (rows - c0)) - 1;     // (no product has the others)
                                    const int skip = skip0 - c0;
                                    if (skip > 0) bits = skip < 32 ? bits >> skip << skip : 0u;
                                    float p4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int c = 0; c < 32; ++c) {
                                        const float p = ex2_approx(fmaf(__uint_as_float(x[c]), a.scale_log2, nl[c0 + c]));
                                        if (bits >> c & 1) p4[c & 3] += p;
                                    }
                                    counted += (p4[0] + p4[1]) + (p4[2] + p4[3]);
                                }
                                if (!plain || again) part = counted;
                            }
                            sum += part;
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(bars->s_empty[w][u]));
                        }
                    }
                    turn ^= 1;
                    if (tiles > 1 || i == g.i1 - 1) {
                        if (lane == 0) mbar_arrive(bar(bars->l_empty[rq.slot]));
                        rq.advance();
                    }
                }
                if (!ok) break;
                if (!sole) {
                    if (u == 1) {
                        ok = wait_warp(wc, bar(bars->x_empty[w][rx.slot]), rx.phase ^ 1, timeout_code(kSiteWXEmpty));
                        if (!ok) break;
                        xch[rx.slot][row] = sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(bars->x_full[w][rx.slot]));
                    } else {
                        ok = wait_warp(wc, bar(bars->x_full[w][rx.slot]), rx.phase, timeout_code(kSiteWXFull));
                        if (!ok) break;
                        sum += xch[rx.slot][row];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(bars->x_empty[w][rx.slot]));
                    }
                    rx.advance();
                }
                if (!owner) continue;
                if (g.whole) {
                    if (key < g.kv) a.out[line + key] = (key < e ? old * a.decay : 0.f) + sum;
                } else {
                    parts[(g.from_start ? kItemKeys : 0) + w * 128 + row] = sum;
                    if (g.from_start && w == 0 && row == 0)
                        cuts[blockIdx.x] = CutItem{g.last_cta, g.seq, g.head, g.i0, e, g.kv, {}};
                }
            }
        }
    }

    __syncthreads();
    if (bars->abort_flag) {
        for (int k = 0; k < 20; ++k) __nanosleep(50000);       // copies and products in flight land
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the parts of the items that were cut, in their order; a thread per key.
__global__ void __launch_bounds__(kItemKeys) paged_weights_join_kernel(const WeightsArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const CutItem cut = reinterpret_cast<const CutItem*>(a.ws + kWeightsParts)[blockIdx.x];
    const int key = cut.item * kItemKeys + (int)threadIdx.x;
    if (cut.last_cta == 0 || key >= cut.kv) return;
    const float* part = reinterpret_cast<const float*>(a.ws) + threadIdx.x;
    const size_t at = ((size_t)cut.seq * a.t.h_kv + cut.head) * a.t.max_pages * a.t.page_size + key;
    const float old = key < cut.old ? a.in[at] * a.decay : 0.f;
    float sum = part[((size_t)blockIdx.x * 2 + 1) * kItemKeys];
    for (int c = (int)blockIdx.x + 1; c <= cut.last_cta; ++c) sum += part[(size_t)c * 2 * kItemKeys];
    a.out[at] = old + sum;
}

size_t weights_ws_bytes() { return kWeightsParts + kPagedMaxCtas * sizeof(CutItem); }

namespace {

template <int D, int ROWS, bool PADDED>
int launch_weights_t(const PagedMaps& m, const WeightsArgs& a, cudaStream_t st)
{
    constexpr uint32_t smem = WeightsCfg<D, ROWS>::SMEM;
    auto kern = paged_weights_kernel<D, ROWS, PADDED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
    const int64_t tiles = ((int64_t)a.t.n_tokens + a.tpt - 1) / a.tpt + a.t.n_seq;
    const int64_t items = ((int64_t)a.t.max_pages * a.t.page_size + kItemKeys - 1) / kItemKeys;
    const int64_t want = tiles * items * a.t.h_kv;
    int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
    if (want < grid) grid = want;
    kern<<<(unsigned)grid, kWeightsThreads, smem, st>>>(m, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return (int)e;
    if (grid > 1 && (int64_t)a.t.n_tokens > (int64_t)(kItemSnap - 1) * a.tpt) {     // else no sequence has items to cut
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(kItemKeys);
        cfg.stream = st;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, paged_weights_join_kernel, a);
    }
    return (int)e;
}

}  // namespace

int weights_tile_rows(const PagedTables& t)
{
    const int64_t group = t.h_q / t.h_kv, items = ((int64_t)t.max_pages * t.page_size + kItemKeys - 1) / kItemKeys;
    // new tokens that make tiles of few rows, on average, and units that 31 bits count
    const bool few = group <= kFewWeightRows && t.n_tokens * group <= (int64_t)kFewWeightRows * t.n_seq &&
                     (t.n_tokens / (kFewWeightRows / group) + 2) * items < INT32_MAX;
    return few ? kFewWeightRows : 128;
}

int launch_weights(const PagedMaps& m, const WeightsArgs& a, cudaStream_t st)
{
    const auto launch = [&](auto head_dim) {
        constexpr int D = decltype(head_dim)::value;
        if (a.rows == kFewWeightRows) return launch_weights_t<D, kFewWeightRows, false>(m, a, st);
        return a.tpt * a.group < a.rows ? launch_weights_t<D, 128, true>(m, a, st)
                                        : launch_weights_t<D, 128, false>(m, a, st);
    };
    switch (a.d) {
        case 64: return launch(std::integral_constant<int, 64>());
        case 96: return launch(std::integral_constant<int, 96>());
        case 128: return launch(std::integral_constant<int, 128>());
        case 160: return launch(std::integral_constant<int, 160>());
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
