// Host check of the work split of the attention over a paged cache
// (attention_core_gb300/csrc/paged_sched.cuh), against counting: for random lengths,
// head groups and CTA counts every block of every tile is in exactly one CTA's share,
// a tile's pieces lie in consecutive CTAs in order, a CTA has at most one piece that
// continues a tile and one that starts one, and the closed-form sums equal the counts.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "../attention_core_gb300/csrc/paged_sched.cuh"

using namespace ac;

static long bad = 0, cuts = 0;
#define WANT(x) (bad += !(x))

static int blocks_by_counting(const SeqShape& s, int m)
{
    int most = 0;
    for (int t = m * s.tpt; t < (m + 1) * s.tpt && t < s.nq; ++t) {
        long seen = s.causal ? (long)s.kv - s.nq + t + 1 : s.kv;
        if (seen > s.kv) seen = s.kv;
        if (seen > 0 && (seen + 127) / 128 > most) most = (int)((seen + 127) / 128);
    }
    return most;
}

static void one()
{
    const int ns = 1 + rand() % 6, h_kv = 1 + rand() % 4, causal = rand() % 4 != 0, ctas = 1 + rand() % 40;
    const int group = rand() % 2 ? 1 << (rand() % 8) : 1 + rand() % 128, tpt = 128 / group;
    const int big = rand() % 3;
    std::vector<int> cu(1, 0), kv;
    for (int i = 0; i < ns; ++i) {
        cu.push_back(cu.back() + (rand() % 3 == 0 ? rand() % 3 : rand() % (big == 2 ? 3000 : 300)));
        kv.push_back(rand() % 5 == 0 ? 0 : rand() % (big ? 5000 : 400));
    }
    PagedTables t{};
    t.cu_q = cu.data();
    t.kv_lens = kv.data();
    t.n_seq = ns;
    t.n_tokens = cu.back();
    t.h_kv = h_kv;
    t.h_q = h_kv * group;
    t.max_pages = 1000;
    t.page_size = 16;
    std::vector<int64_t> first(1, 0);
    int64_t tiles = 0;
    for (int i = 0; i < ns; ++i) {
        const SeqTable q = read_seq(t, i, tpt, causal);
        WANT(!q.bad);
        int64_t sum = 0;
        for (int m = 0; m < q.s.tiles(); ++m) {
            WANT(q.s.units(m) == sum);
            WANT(q.s.blocks(m) == blocks_by_counting(q.s, m));
            sum += q.s.cost(m);
        }
        WANT(q.s.units(q.s.tiles()) == sum);
        first.push_back(first.back() + sum * h_kv);
        tiles += q.s.tiles() * h_kv;
    }
    const int snap = snap_blocks(tiles, ctas);
    const int64_t total = first.back();
    int64_t per = (total + ctas - 1) / ctas;
    if (per < kMinUnits) per = kMinUnits;
    std::map<std::tuple<int, int, int>, std::vector<std::tuple<int, int, int>>> pieces;
    for (int c = 0; c < ctas; ++c) {
        const int64_t u0 = c * per, u1 = u0 + per < total ? u0 + per : total;
        if (u0 >= u1) continue;
        int s = 0;
        while (first[s + 1] <= u0) ++s;
        const SeqTable q = read_seq(t, s, tpt, causal);
        const int64_t head = q.s.units(q.s.tiles()), rel = u0 - first[s];
        SegmentWalk w;
        w.tpt = tpt;
        w.causal = causal;
        w.snap = snap;
        w.start(s, q, (int)(rel / head), (int)(rel % head), u0, u1);
        Segment g;
        int starts = 0, continues = 0;
        while (w.next(t, g)) {
            pieces[{g.seq, g.head, g.m}].push_back({g.j0, g.j1, c});
            WANT(g.n_tok >= 1 && g.q_tok >= cu[g.seq] && g.q_tok + g.n_tok <= cu[g.seq + 1]);
            if (g.whole) continue;
            ++cuts;
            WANT(g.j1 - g.j0 < read_seq(t, g.seq, tpt, causal).s.blocks(g.m));
            WANT(read_seq(t, g.seq, tpt, causal).s.blocks(g.m) > snap);
            if (g.from_start) {
                ++starts;
                const int64_t last = (g.tile_end - 1) / per;
                WANT(last > c && last < ctas);
            } else {
                ++continues;
            }
        }
        WANT(starts <= 1 && continues <= 1);
    }
    for (int i = 0; i < ns; ++i) {
        const SeqTable q = read_seq(t, i, tpt, causal);
        for (int h = 0; h < h_kv; ++h)
            for (int m = 0; m < q.s.tiles(); ++m) {
                const auto& p = pieces[{i, h, m}];
                WANT(!p.empty());
                int at = 0, cta = -1;
                for (const auto& x : p) {
                    WANT(std::get<0>(x) == at && (cta < 0 || std::get<2>(x) == cta + 1));
                    at = std::get<1>(x);
                    cta = std::get<2>(x);
                }
                WANT(at == q.s.blocks(m));
            }
    }
}

int main()
{
    srand(1);
    for (int i = 0; i < 5000; ++i) one();
    // tables that do not fit the tensors make a sequence empty
    const int cu[] = {0, 5, 3, 9, 400}, kv[] = {4, 4, -1, 1 << 30};
    PagedTables t{};
    t.cu_q = cu;
    t.kv_lens = kv;
    t.n_seq = 4;
    t.n_tokens = 100;
    t.h_kv = t.h_q = 1;
    t.max_pages = 8;
    t.page_size = 16;
    WANT(!read_seq(t, 0, 128, 1).bad);
    for (int i = 1; i < 4; ++i) WANT(read_seq(t, i, 128, 1).bad && read_seq(t, i, 128, 1).s.tiles() == 0);
    printf("%ld wrong, %ld cuts\n", bad, cuts);
    return bad != 0 || cuts == 0;
}
