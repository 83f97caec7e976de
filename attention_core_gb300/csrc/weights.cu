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
// Bounds: single tokens the keys' bytes; chunks the exponentials and the product alike.
//
// Persistent, one CTA per SM, equal shares of the work (weights_sched.cuh).  384 threads:
//   warp 3  scheduler: runs of items, in a ring of jobs that the others read
//   warp 0  K, by TMA: an item's 256 keys as two tiles of 128
//   warp 2  row tiles: Q by TMA, and the rows' -LSE log2 e with a bit per row that counts
//           (of a token of the sequence, its LSE not -inf).  A sequence of one tile keeps
//           it for the whole run.
//   warp 1  issues the tcgen05 MMAs: per row tile and half of the item one [128 keys x
//           rows] product, N only as wide as the tile has rows
//   warps 4-11  two warpgroups, each the owner of one half's 128 keys: two TMEM buffers
//           each, exponentials, sums
// A score is fp32; a tile's exponentials are summed in four fp32 chains, and the tiles'
// sums on top, so that thousands of rows lose no more than their tiles' count.
#include <stddef.h>

#include "paged_attn.cuh"
#include "weights_sched.cuh"

namespace ac {

namespace {

template <int D>
struct WeightsCfg {
    static constexpr uint32_t TILE = PagedGeom<D>::TILE;
    static constexpr int SK = D <= 64 ? 8 : D <= 96 ? 5 : 3;       // K tiles
    static constexpr int SQ = D <= 96 ? 4 : D <= 128 ? 3 : 2;      // row tiles
    static constexpr uint32_t OFF_Q = SK * TILE;
    static constexpr uint32_t OFF_BAR = OFF_Q + SQ * TILE;
    static constexpr uint32_t BAR_BYTES = 4096;
    static constexpr uint32_t SMEM = OFF_BAR + BAR_BYTES + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

struct WeightsBars {
    float nlse[4][128];             // a row tile's -LSE log2 e
    uint32_t counts[4][4];          // its rows that count
    uint64_t k_full[8], k_empty[8];
    uint64_t q_full[4], q_empty[4], l_full[4];
    uint64_t s_full[2][2];          // [warpgroup][buffer]
    uint64_t job_full[kJobs];
    uint64_t drain, never;
    uint64_t s_empty[2][2];         // 128 arrivals
    uint64_t l_empty[4];            // kRowThreads
    uint64_t job_empty[kJobs];
    int64_t warp_sum[kThreads / 32];
    ItemWalk walk;
    uint32_t tmem_base;
    int32_t abort_flag;
    ItemRun job[kJobs];
};
static_assert(sizeof(WeightsBars) <= WeightsCfg<64>::BAR_BYTES, "barrier block");
constexpr int kWeightsReaders = 3 + kRowThreads / 32;

enum : int32_t {
    kSiteWInject = 32, kSiteWJobEmpty, kSiteWJobFull, kSiteWKEmpty, kSiteWKFull, kSiteWQEmpty, kSiteWQFull,
    kSiteWLEmpty, kSiteWLFull, kSiteWSEmpty, kSiteWSFull, kSiteWDrain
};

// A cut item, written by the CTA that has its first piece (slot 1 of its own two; the
// later pieces are in slot 0 of the CTAs after it).
struct CutItem {
    int32_t last_cta;    // 0: this CTA cut no item at its end
    int32_t seq, head, item, old, kv;
    int32_t pad[2];
};
constexpr size_t kWeightsParts = (size_t)kPagedMaxCtas * 2 * kItemKeys * sizeof(float);

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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_weights_kernel(const __grid_constant__ PagedMaps maps, const WeightsArgs a)
{
    using P = PagedGeom<D>;
    using C = WeightsCfg<D>;
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
        const int once = (int)(&bars->s_empty[0][0] - first);
        for (int i = lane; i < once; i += 32) mbar_init(bar(first[i]), 1);
        if (lane < 4) mbar_init(bar((&bars->s_empty[0][0])[lane]), 128);
        if (lane < 4) mbar_init(bar(bars->l_empty[lane]), kRowThreads);
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

    // this CTA's share, as in paged_attn.cuh
    const int order = ((int)threadIdx.x + kThreads - 128) % kThreads;     // warp 4 first
    const int run = (t.n_seq + kThreads - 1) / kThreads;
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
    for (int w = 0; w < kThreads / 32; ++w) {
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

    if (alive && warp == 3) {
        Ring<kJobs> jr;
        ItemWalk walk = bars->walk;
        for (bool more = true; more;) {
            if (!wait_w(wc, bar(bars->job_empty[jr.slot]), jr.phase ^ 1, timeout_code(kSiteWJobEmpty))) break;
            ItemRun g;
            more = __all_sync(0xffffffffu, walk.next(t, g));
            if (!more) g.i0 = -1;
            if (lane == 0) {
                bars->job[jr.slot] = g;
                mbar_arrive(bar(bars->job_full[jr.slot]));
            }
            __syncwarp();
            jr.advance();
        }
    } else if (alive && warp == 0) {
        // ---- K: page_table entries 32 at a time, one a lane, the next 32 on their way.  A
        // page outside the cache reads as zeros and is reported.
        const int rows_shift = t.page_shift < 7 ? t.page_shift : 7;
        Ring<C::SK> rk;
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        while (ok && next_run(bars, wc, jr, g)) {
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
        }
    } else if (alive && warp == 2) {
        // ---- row tiles
        int r_tok[4], r_head[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r_tok[k] = (int)(lane + 32 * k) / group;
            r_head[k] = (int)(lane + 32 * k) - r_tok[k] * group;
        }
        Ring<C::SQ> rq;
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        auto load = [&](int m) -> bool {
            const int tok0 = g.q0 + m * tpt;
            const int n_tok = g.nq - m * tpt < tpt ? g.nq - m * tpt : tpt;
            float l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                l[k] = r_tok[k] < n_tok
                           ? a.lse[(size_t)(g.head * group + r_head[k]) * t.n_tokens + tok0 + r_tok[k]] : -INFINITY;
            if (!wait_w(wc, bar(bars->q_empty[rq.slot]), rq.phase ^ 1, timeout_code(kSiteWQEmpty))) return false;
            if (lane == 0) mbar_arrive_expect_tx(bar(bars->q_full[rq.slot]), (uint32_t)(tpt * group) * (D * 2));
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < P::CHUNKS; ++ch)
                tma_load_4d_warp(sb + C::OFF_Q + rq.slot * C::TILE + P::offset(ch), &maps.q[P::narrow(ch)], ch * 64, 0,
                                 g.head, tok0, bar(bars->q_full[rq.slot]));
            if (!wait_w(wc, bar(bars->l_empty[rq.slot]), rq.phase ^ 1, timeout_code(kSiteWLEmpty))) return false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool counts = l[k] != -INFINITY;
                const uint32_t bits = __ballot_sync(0xffffffffu, counts);
                if (lane == 0) bars->counts[rq.slot][k] = bits;
                bars->nlse[rq.slot][lane + 32 * k] = counts ? l[k] * -1.44269504088896340736f : 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bars->l_full[rq.slot]));
            rq.advance();
            return true;
        };
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles();
            if (tiles == 1) {
                ok = load(0);
                continue;
            }
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const int m1 = g.whole ? tiles : g.m1;
                for (int m = g.whole ? s.first_tile(i * kItemKeys) : g.m0; ok && m < m1; ++m) ok = load(m);
            }
        }
    } else if (alive && warp == 1) {
        // ---- MMA issuer: S^T of each half of the item that the tile's rows see
        Ring<C::SK> rk;
        Ring<C::SQ> rq;
        Ring<2> rs[2];
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles();
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const int halves = g.kv - i * kItemKeys > 128 ? 2 : 1;
                Ring<C::SK> rk2 = rk;
                if (halves == 2) rk2.advance();
                const int m1 = g.whole ? tiles : g.m1;
                const int sees2 = halves == 2 ? s.first_tile(i * kItemKeys + 128) : INT32_MAX;
                int m = g.whole ? s.first_tile(i * kItemKeys) : g.m0;
                const int first = m;
                bool waited2 = false;
                for (; ok && m < m1; ++m) {
                    const bool last_use = tiles > 1 || i == g.i1 - 1;
                    if (tiles > 1 || i == g.i0)
                        ok = wait_w(wc, bar(bars->q_full[rq.slot]), rq.phase, timeout_code(kSiteWQFull));
                    if (!ok) break;
                    const int rows = (g.nq - m * tpt < tpt ? g.nq - m * tpt : tpt) * group;
                    const uint32_t ids = idesc_bf16(128, 0, false, false) | (uint32_t)((rows + 15) / 16 * 2) << 17;
                    const uint32_t qbase = sb + C::OFF_Q + rq.slot * C::TILE;
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
                        if (w == 1 && m < sees2) break;
                        const Ring<C::SK>& r = w ? rk2 : rk;
                        if (w ? !waited2 : m == first)
                            ok = wait_w(wc, bar(bars->k_full[r.slot]), r.phase, timeout_code(kSiteWKFull));
                        waited2 |= w == 1;
                        Ring<2>& b = rs[w];
                        ok = ok && wait_w(wc, bar(bars->s_empty[w][b.slot]), b.phase ^ 1, timeout_code(kSiteWSEmpty));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t tS = tmem + (uint32_t)(w * 2 + b.slot) * 128;
                        const uint32_t kbase = sb + r.slot * C::TILE;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tS, P::desc_k(kbase, kk), P::desc_k(qbase, kk), ids, kk > 0 ? 1u : 0u);
                        mma_commit(bar(bars->s_full[w][b.slot]));
                        b.advance();
                    }
                    if (!ok) break;
                    if (last_use) {
                        mma_commit(bar(bars->q_empty[rq.slot]));
                        rq.advance();
                    }
                }
                if (!ok) break;
                // (a second half that no tile of a piece sees has to land before its slot is free)
                if (halves == 2 && !waited2)
                    ok = wait_w(wc, bar(bars->k_full[rk2.slot]), rk2.phase, timeout_code(kSiteWKFull));
                if (!ok) break;
                mma_commit(bar(bars->k_empty[rk.slot]));
                rk.advance();
                if (halves == 2) {
                    mma_commit(bar(bars->k_empty[rk.slot]));
                    rk.advance();
                }
            }
        }
        mma_commit(bar(bars->drain));
        wait_w(wc, bar(bars->drain), 0, timeout_code(kSiteWDrain));
    } else if (alive && warp >= 4) {
        // ---- sums: a thread per key of its warpgroup's half
        const RowThread rt = row_thread();
        const int w = rt.half;
        Ring<C::SQ> rq;
        Ring<2> rs;
        Ring<kJobs> jr;
        ItemRun g{};
        bool ok = true;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
        const size_t length = (size_t)t.max_pages * t.page_size;
        while (ok && next_run(bars, wc, jr, g)) {
            const ItemShape s = shape(g);
            const int tiles = s.tiles(), e = g.kv - g.nq;
            const size_t line = ((size_t)g.seq * t.h_kv + g.head) * length;
            for (int i = g.i0; ok && i < g.i1; ++i) {
                const int key0 = i * kItemKeys + w * 128, key = key0 + rt.row;
                const int m1 = g.whole ? tiles : g.m1;
                const int sees = key0 < g.kv ? s.first_tile(key0) : INT32_MAX;
                float old = 0.f, sum = 0.f;
                if (g.whole && key < e) old = a.in[line + key];
                for (int m = g.whole ? s.first_tile(i * kItemKeys) : g.m0; m < m1; ++m) {
                    if (tiles > 1 || i == g.i0)
                        ok = wait_warp(wc, bar(bars->l_full[rq.slot]), rq.phase, timeout_code(kSiteWLFull));
                    if (!ok) break;
                    if (m >= sees) {
                        ok = wait_warp(wc, bar(bars->s_full[w][rs.slot]), rs.phase, timeout_code(kSiteWSFull));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t tS = tmem + (uint32_t)(w * 2 + rs.slot) * 128 + rt.lane_off;
                        const float* nl = bars->nlse[rq.slot];
                        const uint4 counts = *reinterpret_cast<const uint4*>(bars->counts[rq.slot]);
                        const int pos = e + m * tpt;                        // of the tile's first token
                        if ((counts.x & counts.y & counts.z & counts.w) == 0xffffffffu &&
                            (!a.causal || key0 + 127 <= pos)) {
                            uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t x[64];
                                tmem_ld64(tS + 64 * half, x);
#pragma unroll
                                for (int c = 0; c < 64; c += 4) {
                                    const float4 n4 = *reinterpret_cast<const float4*>(nl + 64 * half + c);
                                    float lo, hi;
                                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2,
                                                     f2_pack(n4.x, n4.y)), lo, hi);
                                    acc[c / 4 * 2 & 3] = f2_add(acc[c / 4 * 2 & 3], f2_pack(ex2_approx(lo), ex2_approx(hi)));
                                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2,
                                                     f2_pack(n4.z, n4.w)), lo, hi);
                                    acc[(c / 4 * 2 + 1) & 3] =
                                        f2_add(acc[(c / 4 * 2 + 1) & 3], f2_pack(ex2_approx(lo), ex2_approx(hi)));
                                }
                            }
                            float lo, hi;
                            f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
                            sum += lo + hi;
                        } else {
                            // rows that do not count, or whose mask hides this key, are left out
                            // whatever their score is
                            const int rows = (g.nq - m * tpt < tpt ? g.nq - m * tpt : tpt) * group;
                            const int from = a.causal && key > pos ? (key - pos) * group : 0;
                            float part = 0.f;
#pragma unroll 1
                            for (int c0 = 0; c0 < rows; c0 += 32) {
                                uint32_t x[32];
                                tmem_ld32(tS + c0, x);
                                uint32_t bits = bars->counts[rq.slot][c0 / 32];
                                const int skip = from - c0;
                                if (skip > 0) bits = skip < 32 ? bits >> skip << skip : 0u;
                                float p4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int c = 0; c < 32; ++c) {
                                    const float p = ex2_approx(fmaf(__uint_as_float(x[c]), a.scale_log2, nl[c0 + c]));
                                    if (bits >> c & 1) p4[c & 3] += p;
                                }
                                part += (p4[0] + p4[1]) + (p4[2] + p4[3]);
                            }
                            sum += part;
                        }
                        tc_fence_before();
                        mbar_arrive(bar(bars->s_empty[w][rs.slot]));
                        rs.advance();
                    }
                    if (tiles > 1 || i == g.i1 - 1) {
                        mbar_arrive(bar(bars->l_empty[rq.slot]));
                        rq.advance();
                    }
                }
                if (!ok) break;
                if (g.whole) {
                    if (key < g.kv) a.out[line + key] = (key < e ? old * a.decay : 0.f) + sum;
                } else {
                    parts[(g.from_start ? kItemKeys : 0) + w * 128 + rt.row] = sum;
                    if (g.from_start && w == 0 && rt.row == 0)
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

template <int D>
int launch_weights_t(const PagedMaps& m, const WeightsArgs& a, cudaStream_t st)
{
    constexpr uint32_t smem = WeightsCfg<D>::SMEM;
    auto kern = paged_weights_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
    const int64_t tiles = ((int64_t)a.t.n_tokens + a.tpt - 1) / a.tpt + a.t.n_seq;
    const int64_t items = ((int64_t)a.t.max_pages * a.t.page_size + kItemKeys - 1) / kItemKeys;
    const int64_t want = tiles * items * a.t.h_kv;
    int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
    if (want < grid) grid = want;
    kern<<<(unsigned)grid, kThreads, smem, st>>>(m, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return (int)e;
    if (grid > 1 && (int64_t)a.t.n_tokens > (int64_t)kItemSnap * a.tpt) {     // else no sequence has items to cut
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

int launch_weights(const PagedMaps& m, const WeightsArgs& a, cudaStream_t st)
{
    switch (a.d) {
        case 64: return launch_weights_t<64>(m, a, st);
        case 96: return launch_weights_t<96>(m, a, st);
        case 128: return launch_weights_t<128>(m, a, st);
        case 160: return launch_weights_t<160>(m, a, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
