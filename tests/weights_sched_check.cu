// Host check of the work split of the gathered attention weights
// (attention_core_gb300/csrc/weights_sched.cuh), against counting: every (item, row
// tile) pair whose rows see the item is in exactly one CTA's share, an item's pieces
// lie in consecutive CTAs in order, a CTA has at most one piece that continues an item
// and one that starts one, and the closed-form sums equal the counts.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "../attention_core_gb300/csrc/weights_sched.cuh"

using namespace ac;

static long bad = 0, cuts = 0;
#define WANT(x) (bad += !(x))

static bool sees(const ItemShape& s, int m, int key)
{
    const long last = (long)(m + 1) * s.tpt < s.nq ? (long)(m + 1) * s.tpt - 1 : s.nq - 1;
    return !s.causal || s.kv - s.nq + last >= key;
}

static void one()
{
    const int ns = 1 + rand() % 6, h_kv = 1 + rand() % 4, causal = rand() % 4 != 0, ctas = 1 + rand() % 40;
    const int group = rand() % 2 ? 1 << (rand() % 8) : 1 + rand() % 128, tpt = 128 / group;
    const int big = rand() % 3;
    std::vector<int> cu(1, 0), kv;
    for (int i = 0; i < ns; ++i) {
        cu.push_back(cu.back() + (rand() % 3 == 0 ? rand() % 3 : rand() % (big == 2 ? 3000 : 300)));
        kv.push_back(rand() % 5 == 0 ? 0 : rand() % (big ? 9000 : 400));
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
    for (int i = 0; i < ns; ++i) {
        const ItemShape s = item_shape(read_seq(t, i, tpt, causal));
        int64_t sum = 0;
        for (int k = 0; k < s.items(); ++k) {
            WANT(s.units(k) == sum);
            WANT(s.cost(k) >= 2);
            for (int j = k * kItemKeys; j < s.kv && j < (k + 1) * kItemKeys; j += 1 + rand() % 60) {
                const int m0 = s.first_tile(j);
                WANT(m0 < s.tiles() && sees(s, m0, j) && (m0 == 0 || !sees(s, m0 - 1, j)));
            }
            sum += s.cost(k);
        }
        WANT(s.units(s.items()) == sum);
        first.push_back(first.back() + sum * h_kv);
    }
    const int64_t total = first.back();
    int64_t per = (total + ctas - 1) / ctas;
    if (per < 1) per = 1;
    std::map<std::tuple<int, int, int>, std::vector<std::tuple<int, int, int>>> pieces;
    for (int c = 0; c < ctas; ++c) {
        const int64_t u0 = c * per, u1 = u0 + per < total ? u0 + per : total;
        if (u0 >= u1) continue;
        int s = 0;
        while (first[s + 1] <= u0) ++s;
        const SeqTable q = read_seq(t, s, tpt, causal);
        const ItemShape sh = item_shape(q);
        const int64_t head = sh.units(sh.items()), rel = u0 - first[s];
        ItemWalk w;
        w.tpt = tpt;
        w.causal = causal;
        w.per = per;
        w.start(s, q, (int)(rel / head), (int)(rel % head), u0, u1);
        ItemRun g;
        int starts = 0, continues = 0;
        while (w.next(t, g)) {
            const ItemShape x = item_shape(read_seq(t, g.seq, tpt, causal));
            WANT(x.nq == g.nq && x.kv == g.kv && g.q0 == cu[g.seq] && g.i1 > g.i0 && g.i1 <= x.items());
            if (g.whole) {
                for (int i = g.i0; i < g.i1; ++i)
                    pieces[{g.seq, g.head, i}].push_back({x.first_tile(i * kItemKeys), x.tiles(), c});
                continue;
            }
            WANT(g.i1 == g.i0 + 1 && g.m1 > g.m0);
            pieces[{g.seq, g.head, g.i0}].push_back({g.m0, g.m1, c});
            ++cuts;
            WANT(x.cost(g.i0) > kItemSnap && g.m1 - g.m0 < x.tiles() - x.first_tile(g.i0 * kItemKeys));
            if (g.from_start) {
                ++starts;
                WANT(g.last_cta > c && g.last_cta < ctas);
            } else {
                ++continues;
            }
        }
        WANT(starts <= 1 && continues <= 1);
    }
    for (int i = 0; i < ns; ++i) {
        const ItemShape s = item_shape(read_seq(t, i, tpt, causal));
        for (int h = 0; h < h_kv; ++h)
            for (int k = 0; k < s.items(); ++k) {
                const auto& p = pieces[{i, h, k}];
                WANT(!p.empty());
                int at = s.first_tile(k * kItemKeys), cta = -1;
                for (const auto& x : p) {
                    WANT(std::get<0>(x) == at && (cta < 0 || std::get<2>(x) == cta + 1));
                    at = std::get<1>(x);
                    cta = std::get<2>(x);
                }
                WANT(at == s.tiles());
            }
    }
}

int main()
{
    srand(1);
    for (int i = 0; i < 5000; ++i) one();
    printf("%ld wrong, %ld cuts\n", bad, cuts);
    return bad != 0 || cuts == 0;
}
