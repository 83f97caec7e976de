// paged_sched.cuh -- work split of the attention over a paged cache.
//
// A tile is up to 128 rows -- `tpt` new tokens times the `group` query heads of
// one KV head -- of one sequence, and its work is the blocks of 128 keys that
// its last row sees (one unit at least: a tile that sees no key still has zeros
// to write).  All tiles, in the order (sequence, KV head, row tile), form one
// line of T units, and CTA c takes the units [c * per, (c + 1) * per), per =
// ceil(T / grid): every CTA gets the same number of blocks whatever the lengths
// are, and a tile is cut only where a CTA's share ends.  The parts of a cut tile
// are joined by a second kernel.  Short tiles are not cut: the CTA whose share holds
// a tile's first unit takes all of it (cutting one costs more, in the join, than the
// imbalance of a few blocks).  How short goes by the tiles (snap_blocks).
//
// The other split hands out whole tiles to whichever CTA is ready for one (a counter
// in the workspace): 32 sequences at a time, those with the most keys first, and of
// each KV head the last row tile first, so that the tiles that go out last are short.
// Nothing is cut and joined, and neighbouring CTAs visit the same keys at the same
// time, which matters where a KV head has several row tiles and the keys of all heads
// do not fit L2; but the last tiles leave CTAs without work.  hand_out_tiles() chooses.
//
// Lengths are device data, so every CTA finds its share by itself: a block-wide
// sum over the sequences' units (closed form under the causal mask), then a walk
// from its first unit on.
#pragma once
#include <stdint.h>

#include "kernels.h"

namespace ac {

constexpr int kMinUnits = 2;    // least share of a CTA
constexpr int kLeastSnap = 4;
// Tiles of at most this many blocks stay whole: few tiles have to be shared out, many
// go round by themselves.  Measured at 4 and 8 (64/8 heads, a single token each): one
// sequence of 1000 keys (8 tiles of 8 blocks) 10.0 and 11.8 us, 16 of 1000 keys 21.4 and
// 17.9, 64 of 700 keys 39.3 and 38.6; a least share of 1 or 4 instead of 2 is within 3%
// or slower.
__host__ __device__ inline int snap_blocks(int64_t tiles, int64_t ctas) { return 2 * tiles >= ctas ? 8 : kLeastSnap; }

// a / b in the 32-bit divide where both fit (nearly always), which takes a
// fraction of the 64-bit one's time
__host__ __device__ inline int64_t quot(int64_t a, int64_t b)
{
    if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
    return (int64_t)((uint32_t)a / (uint32_t)b);
}

// sum over i = 0 .. n - 1 of floor((a i + b) / m), m > 0, where the sum and
// a n + b fit 32 bits (no partial sum is larger)
__host__ __device__ inline uint32_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b)
{
    uint32_t s = 0;
    while (n > 0) {
        const uint32_t qa = a / m, qb = b / m;
        if (qa) s += (n - 1) * n / 2 * qa;
        s += n * qb;
        a -= qa * m;
        b -= qb * m;
        if (a == 0) break;
        const uint32_t top = a * n + b;
        n = top / m;
        b = top - n * m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return s;
}

// One sequence's shape: nq new tokens, kv keys (both below 2^31 - 256), tiles of
// tpt tokens.  The units of one KV head fit 31 bits (the caller sees to it).
struct SeqShape {
    int nq, kv, tpt, causal;
    __host__ __device__ int tiles() const { return (int)(((uint32_t)nq + tpt - 1) / (uint32_t)tpt); }
    // blocks of 128 keys that tile m sees: those of its last row
    __host__ __device__ int blocks(int m) const
    {
        int last = kv;
        if (causal) {
            const int end = kv - nq + (m + 1) * tpt;
            last = end < kv ? end : kv;
        }
        return last <= 0 ? 0 : (int)(((uint32_t)last + 127) / 128);
    }
    __host__ __device__ int cost(int m) const
    {
        const int n = blocks(m);
        return n > 0 ? n : 1;
    }
    // units of the tiles 0 .. m - 1
    __host__ __device__ int units(int m) const;
};

// One copy, by value: instructions are fetched cold at a kernel's start, and
// inlining this at each use made them the largest part of it.
#ifdef __CUDA_ARCH__
__noinline__
#endif
__host__ __device__ inline int units_before(int m, int nq, int kv, int tpt, int causal)
{
    const SeqShape q{nq, kv, tpt, causal};
    if (m <= 0) return 0;
    if (kv <= 0) return m;
    if (!causal) return m * q.cost(0);
    const int e = kv - nq;                                   // keys before the first new token
    const int last = q.tiles() - 1;                          // sees kv keys, however many rows it has
    int z = e < 0 ? (int)((uint32_t)-e / (uint32_t)tpt) : 0; // tiles that see nothing: one unit each
    if (z > m) z = m;
    const int plain = (m < last ? m : last) - z;             // tiles that see e + (i + 1) tpt keys
    uint32_t s = z;
    if (plain > 0) s += floor_sum(plain, 128, tpt, e + (z + 1) * tpt + 127);
    if (m > last) s += q.cost(last);
    return (int)s;
}
__host__ __device__ inline int SeqShape::units(int m) const { return units_before(m, nq, kv, tpt, causal); }

// The last row tile of a head that starts at or before unit r of it.  On the
// device a whole warp calls this with one r: each round its lanes test 32
// candidates.
__host__ __device__ inline int find_tile(const SeqShape& s, int r)
{
    int lo = 0, hi = s.tiles();
    while (hi - lo > 1) {
#ifdef __CUDA_ARCH__
        const int step = (hi - lo + 31) / 32;
        const int m = lo + (int)(threadIdx.x & 31) * step;
        const uint32_t le = __ballot_sync(0xffffffffu, m < hi && s.units(m) <= r);
        lo += (31 - __clz(le)) * step;                       // lane 0's test holds
        hi = lo + step < hi ? lo + step : hi;
#else
        const int m = lo + (hi - lo) / 2;
        (s.units(m) <= r ? lo : hi) = m;
#endif
    }
    return lo;
}

// A sequence as the tables give it, made safe: lengths that do not fit the
// tensors make it empty (`bad`).
struct SeqTable {
    int q0;
    SeqShape s;
    bool bad;
};
__host__ __device__ inline SeqTable read_seq(const PagedTables& t, int seq, int tpt, int causal)
{
    SeqTable r;
    const int q0 = t.cu_q[seq], q1 = t.cu_q[seq + 1], kv = t.kv_lens[seq];
    r.bad = q0 < 0 || q1 < q0 || q1 > t.n_tokens || kv < 0 || kv > (int64_t)t.max_pages * t.page_size;
    r.q0 = q0;
    r.s = SeqShape{r.bad ? 0 : q1 - q0, r.bad ? 0 : kv, tpt, causal};
    return r;
}

// A piece of one tile: blocks [j0, j1) of it.
struct Segment {
    int seq, head, m;      // sequence, KV head, row tile
    int q_tok, n_tok;      // first token (row of q) and tokens of the tile
    int kv;                // keys of the sequence
    int first_pos;         // position of the tile's first token (negative: no key for it)
    int j0, j1;            // blocks of this piece; both 0: the tile sees no key
    int whole;             // the whole tile
    int from_start;        // the tile's first unit is in it
    int last_cta;          // a cut tile's first piece: the CTA of its last one
    int64_t tile_end;      // unit after the tile's last
};

// Tile m of a KV head's, whole.
__host__ __device__ inline Segment whole_tile(const SeqTable& s, int seq, int head, int m)
{
    Segment g;
    g.seq = seq;
    g.head = head;
    g.m = m;
    g.q_tok = s.q0 + m * s.s.tpt;
    g.n_tok = s.s.nq - m * s.s.tpt < s.s.tpt ? s.s.nq - m * s.s.tpt : s.s.tpt;
    g.kv = s.s.kv;
    g.first_pos = s.s.kv - s.s.nq + m * s.s.tpt;
    g.j0 = 0;
    g.j1 = s.s.blocks(m);
    g.whole = g.from_start = 1;
    g.last_cta = 0;
    g.tile_end = 0;
    return g;
}

// Walks a CTA's share of the line.  `at` is the unit at which the next segment
// starts; the CTA's share ends at `end`.
struct SegmentWalk {
    int tpt, causal, snap;
    int64_t at, end;
    int seq, head, m, b;   // where `at` is: block b of row tile m
    SeqTable cur;

    __host__ __device__ void load(const PagedTables& t) { cur = read_seq(t, seq, tpt, causal); }

    // Unit `at_` lies r units into KV head h of sequence sq.  (Whole warps, see
    // find_tile.)
    __host__ __device__ void start(int sq, const SeqTable& table, int h, int r, int64_t at_, int64_t end_)
    {
        at = at_;
        end = end_;
        seq = sq;
        cur = table;
        head = h;
        m = find_tile(cur.s, r);
        b = r - cur.s.units(m);
        const int n = cur.s.cost(m);
        if (b > 0 && n <= snap) {                           // another CTA has all of this tile
            at += n - b;
            b = n;
        }
    }

    __host__ __device__ bool next(const PagedTables& t, Segment& g)
    {
        if (at >= end) return false;
        int n = cur.s.cost(m);
        if (b >= n) {
            b = 0;
            if (++m >= cur.s.tiles()) {
                m = 0;
                if (++head >= t.h_kv) {
                    head = 0;
                    do {
                        if (++seq >= t.n_seq) {              // only past the line's end
                            at = end;
                            return false;
                        }
                        load(t);
                    } while (cur.s.nq <= 0);
                }
            }
            n = cur.s.cost(m);
        }
        const int64_t left = end - at;
        const int take = (n <= snap || left > n - b) ? n - b : (int)left;
        g = whole_tile(cur, seq, head, m);
        const bool sees = cur.s.blocks(m) > 0;
        g.j0 = sees ? b : 0;
        g.j1 = sees ? b + take : 0;
        g.whole = take == n;
        g.from_start = b == 0;
        g.tile_end = at + (n - b);
        at += take;
        b += take;
        return true;
    }
};

}  // namespace ac
