// weights_sched.cuh -- work split of the attention weights gathered by a cache's keys.
//
// An item is 256 keys of one sequence and KV head, and its work the load of the keys, one
// unit, and one for each row tile (`tpt` new tokens times the head group) that sees its
// first key; every item of a sequence with new tokens has one such tile at least, the last
// row's.  (Without the loads' unit, CTAs with single tokens were busy for 42 us where
// those with chunks were done after 27: eight sequences, 16 heads of 160.)  All units, in
// the order (sequence, KV head, item, load and tiles), form one line, and CTA c takes the
// units [c * per, (c + 1) * per): an item is cut only where a share ends, and the parts'
// sums are added by a second kernel.  Items of few units stay whole, in the CTA whose
// share holds their first unit, and no piece is a load alone.
#pragma once
#include "paged_sched.cuh"

namespace ac {

constexpr int kItemKeys = 256;
constexpr int kItemSnap = 5;      // items of at most this many units (four tiles) are not cut

// units of the items 0 .. i - 1 of one KV head (they fit 31 bits, as paged_sched.cuh's)
#ifdef __CUDA_ARCH__
__noinline__
#endif
__host__ __device__ inline int item_units(int i, int nq, int kv, int tpt, int causal)
{
    const int tiles = (int)(((uint32_t)nq + tpt - 1) / (uint32_t)tpt);
    if (!causal) return i * (tiles + 1);
    const int e = kv - nq;                                        // keys before the first new token
    const int from = e > 0 ? (int)(((uint32_t)e + kItemKeys - 1) / kItemKeys) : 0;   // items before are seen by all tiles
    if (i <= from) return i * (tiles + 1);
    return i * (tiles + 1) - (int)floor_sum((uint32_t)(i - from), (uint32_t)tpt, kItemKeys, (uint32_t)(from * kItemKeys - e));
}

struct ItemShape {
    int nq, kv, tpt, causal;
    __host__ __device__ int tiles() const { return (int)(((uint32_t)nq + tpt - 1) / (uint32_t)tpt); }
    __host__ __device__ int items() const { return nq > 0 ? (int)(((uint32_t)kv + kItemKeys - 1) / kItemKeys) : 0; }
    // first row tile that sees key j (0 <= j < kv)
    __host__ __device__ int first_tile(int j) const
    {
        const int e = kv - nq;
        return !causal || j <= e ? 0 : (int)((uint32_t)(j - e) / (uint32_t)tpt);
    }
    __host__ __device__ int cost(int i) const { return 1 + tiles() - first_tile(i * kItemKeys); }
    __host__ __device__ int units(int i) const { return item_units(i, nq, kv, tpt, causal); }
};
__host__ __device__ inline ItemShape item_shape(const SeqTable& q) { return ItemShape{q.s.nq, q.s.kv, q.s.tpt, q.s.causal}; }

// The last item of a head that starts at or before unit r of it (whole warps on the
// device, as find_tile).
__host__ __device__ inline int find_item(const ItemShape& s, int r)
{
    int lo = 0, hi = s.items();
    while (hi - lo > 1) {
#ifdef __CUDA_ARCH__
        const int step = (hi - lo + 31) / 32;
        const int m = lo + (int)(threadIdx.x & 31) * step;
        const uint32_t le = __ballot_sync(0xffffffffu, m < hi && s.units(m) <= r);
        lo += (31 - __clz(le)) * step;
        hi = lo + step < hi ? lo + step : hi;
#else
        const int m = lo + (hi - lo) / 2;
        (s.units(m) <= r ? lo : hi) = m;
#endif
    }
    return lo;
}

// A run of whole items, or a piece of one: the tiles [m0, m1) of item i0.
struct ItemRun {
    int seq, head;
    int q0, nq, kv;
    int i0, i1;
    int whole;
    int m0, m1;            // of a piece
    int from_start;        // a piece that holds the item's first unit
    int last_cta;          // of such a piece: the CTA of the item's last one
};

struct ItemWalk {
    int tpt, causal;
    int64_t at, end, per;
    int seq, head, i, b;   // where `at` is: unit b of item i
    int line_b;            // 1: `at` is a unit further than b
    SeqTable cur;

    // Unit `at_` lies r units into KV head h of sequence sq.  (Whole warps.)
    __host__ __device__ void start(int sq, const SeqTable& table, int h, int r, int64_t at_, int64_t end_)
    {
        at = at_;
        end = end_;
        seq = sq;
        cur = table;
        head = h;
        line_b = 0;
        const ItemShape s = item_shape(cur);
        i = find_item(s, r);
        const int n = s.cost(i);
        b = r - s.units(i);
        if (b > 0 && n <= kItemSnap) {                      // another CTA has all of this item
            at += n - b;
            b = n;
        } else if (b == 1) {
            b = 0;                                          // and none just the load of it
            line_b = 1;
        }
    }

    __host__ __device__ bool next(const PagedTables& t, ItemRun& g)
    {
        if (at >= end) return false;
        ItemShape s = item_shape(cur);
        int n = s.cost(i);
        if (b >= n) {                                       // on to the next item
            if (++i >= s.items()) {
                i = 0;
                if (++head >= t.h_kv) {
                    head = 0;
                    do {
                        if (++seq >= t.n_seq) {             // only past the line's end
                            at = end;
                            return false;
                        }
                        cur = read_seq(t, seq, tpt, causal);
                        s = item_shape(cur);
                    } while (s.items() <= 0);
                }
            }
            b = 0;
            n = s.cost(i);
        }
        g.seq = seq;
        g.head = head;
        g.q0 = cur.q0;
        g.nq = s.nq;
        g.kv = s.kv;
        g.i0 = i;
        g.last_cta = 0;
        g.from_start = b == 0;
        const int skipped = line_b;        // this item's first unit is in the share before
        line_b = 0;
        if (g.from_start && (n <= kItemSnap || n - skipped <= end - at)) {
            // whole items, as many as are this CTA's
            g.whole = 1;
            g.m0 = g.m1 = 0;
            at -= skipped;
            for (;;) {
                at += n;
                if (i + 1 >= s.items() || at >= end) break;
                const int next = s.cost(i + 1);
                if (next > kItemSnap && next > end - at) break;
                ++i;
                n = next;
            }
            g.i1 = i + 1;
            b = n;
            return true;
        }
        const int64_t left = end - at;
        if (g.from_start && left + skipped == 1) {
            at = end;
            return false;
        }
        const int take = left + skipped < n - b ? (int)left + skipped : n - b;
        const int first = s.tiles() - n + 1;                // the item's first tile
        g.whole = 0;
        g.i1 = i + 1;
        g.m0 = b > 0 ? first + b - 1 : first;
        g.m1 = first + b + take - 1;
        if (g.from_start) g.last_cta = (int)quot(at - skipped + n - 1, per);
        at += take - skipped;
        b += take;
        return true;
    }
};

}  // namespace ac
