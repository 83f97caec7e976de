// rope.cu -- rotary positions on sm_103a: the rotation of Q and K (and of their
// gradients), and the append of new tokens to a paged key/value cache with the
// rotation fused in.
//
// Pair (x_a, x_b) of a head turns by w = position * f_i.  The frequency comes
// as a 64-bit fraction of a turn per position, so position * turns[i] modulo
// 2^64 is the angle reduced exactly at any position (a product in fp32 is off
// by 0.06 rad at position 10^6); its top 32 bits, as a signed fraction of a
// turn, go to sincospi.  Arithmetic is fp32, rounded once to bf16.
//
// Both kernels are bound by HBM: every element is read and written once.  A
// thread owns one 16-byte unit of pairs of one token, keeps its cosines and
// sines in registers and walks over some of the heads, so an angle is formed
// once for all of those and there is no shared memory; the first heads' loads go
// out before the angles are formed.  Measured: Q and K of [1, 64 + 8, 8192, 128]
// 45.8 us (6.6 TB/s, 97% of a plain copy's rate; 54.0 with all heads in one block and
// loads behind the angles), [2, 12 + 12, 2048, 128] with half of each head 11.1 us (a
// plain copy of the same bytes: 9.1), the tiny [1, 2 + 2, 128, 64] 2.5 us, all in a
// graph; single calls of the last one take the host's 11 us.
#include "kernels.h"
#include "ptx.cuh"

namespace ac {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kAhead = 4;   // heads of a thread: the loads that it has in flight

__device__ __forceinline__ uint32_t rot_pair16(uint32_t xa, uint32_t xb, float c0, float s0, float c1, float s1,
                                               uint32_t& yb)
{
    const float a0 = __uint_as_float(xa << 16), a1 = __uint_as_float(xa & 0xffff0000u);
    const float b0 = __uint_as_float(xb << 16), b1 = __uint_as_float(xb & 0xffff0000u);
    yb = pack_bf16x2(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
    return pack_bf16x2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
}

// How a row's units are laid out: MODE 0 pairs (i, i + rot / 2), 8 pairs a unit
// (rot % 16 == 0); MODE 1 the same with 4 pairs a unit (rot % 16 == 8, whose
// second halves are only 8-byte aligned); MODE 2 interleaved, 4 pairs a unit.
// Units past the pairs copy 8 values each.
template <int MODE>
struct Unit {
    static constexpr int PAIRS = MODE == 0 ? 8 : 4;
    float c[PAIRS], s[PAIRS];
    int u, n_pair_units, half, rot;

    __device__ __forceinline__ void place(const RopeTable& t, int unit)
    {
        u = unit;
        rot = t.rot;
        half = t.rot / 2;
        n_pair_units = half / PAIRS;
    }
    __device__ __forceinline__ void turn(const RopeTable& t, int64_t pos, float sign)
    {
        if (u >= n_pair_units) return;
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const uint64_t turn = (uint64_t)pos * t.turns[u * PAIRS + e];
            // signed fraction of a turn in [-1/2, 1/2), doubled: sincospi's half turns
            const float x = (float)(int32_t)(turn >> 32) * 0x1p-31f;
            float sn, cs;
            sincospif(x, &sn, &cs);
            c[e] = cs * t.mscale;
            s[e] = sn * (t.mscale * sign);
        }
    }
    struct Data {
        uint4 a, b;
    };
    __device__ __forceinline__ Data load(const uint16_t* row) const
    {
        Data d;
        d.b = make_uint4(0u, 0u, 0u, 0u);
        if (u >= n_pair_units) {
            d.a = *reinterpret_cast<const uint4*>(row + rot + (u - n_pair_units) * 8);
        } else if (MODE == 0) {
            d.a = *reinterpret_cast<const uint4*>(row + u * 8);
            d.b = *reinterpret_cast<const uint4*>(row + half + u * 8);
        } else if (MODE == 1) {
            const uint2 lo = *reinterpret_cast<const uint2*>(row + u * 4);
            const uint2 hi = *reinterpret_cast<const uint2*>(row + half + u * 4);
            d.a = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            d.a = *reinterpret_cast<const uint4*>(row + u * 8);
        }
        return d;
    }
    // the values as they are (no product with 1: an infinity would reach its partner)
    __device__ __forceinline__ void store_raw(uint16_t* row, const Data& d) const
    {
        if (u >= n_pair_units) {
            *reinterpret_cast<uint4*>(row + rot + (u - n_pair_units) * 8) = d.a;
        } else if (MODE == 0) {
            *reinterpret_cast<uint4*>(row + u * 8) = d.a;
            *reinterpret_cast<uint4*>(row + half + u * 8) = d.b;
        } else if (MODE == 1) {
            *reinterpret_cast<uint2*>(row + u * 4) = make_uint2(d.a.x, d.a.y);
            *reinterpret_cast<uint2*>(row + half + u * 4) = make_uint2(d.a.z, d.a.w);
        } else {
            *reinterpret_cast<uint4*>(row + u * 8) = d.a;
        }
    }
    __device__ __forceinline__ void store(uint16_t* row, const Data& d) const
    {
        if (u >= n_pair_units) {
            *reinterpret_cast<uint4*>(row + rot + (u - n_pair_units) * 8) = d.a;
        } else if constexpr (MODE == 0) {
            uint4 a, b;
            a.x = rot_pair16(d.a.x, d.b.x, c[0], s[0], c[1], s[1], b.x);
            a.y = rot_pair16(d.a.y, d.b.y, c[2], s[2], c[3], s[3], b.y);
            a.z = rot_pair16(d.a.z, d.b.z, c[4], s[4], c[5], s[5], b.z);
            a.w = rot_pair16(d.a.w, d.b.w, c[6], s[6], c[7], s[7], b.w);
            *reinterpret_cast<uint4*>(row + u * 8) = a;
            *reinterpret_cast<uint4*>(row + half + u * 8) = b;
        } else if constexpr (MODE == 1) {
            uint2 a, b;
            a.x = rot_pair16(d.a.x, d.a.z, c[0], s[0], c[1], s[1], b.x);
            a.y = rot_pair16(d.a.y, d.a.w, c[2], s[2], c[3], s[3], b.y);
            *reinterpret_cast<uint2*>(row + u * 4) = a;
            *reinterpret_cast<uint2*>(row + half + u * 4) = b;
        } else {
            const uint32_t w[4] = {d.a.x, d.a.y, d.a.z, d.a.w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float xa = __uint_as_float(w[e] << 16), xb = __uint_as_float(w[e] & 0xffff0000u);
                y[e] = pack_bf16x2(xa * c[e] - xb * s[e], xb * c[e] + xa * s[e]);
            }
            *reinterpret_cast<uint4*>(row + u * 8) = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
};

__host__ __device__ inline int units_of(int mode, int d, int rot)
{
    return rot / (mode == 0 ? 16 : 8) + (d - rot) / 8;
}

}  // namespace

// One block: `tile` tokens of one batch element and, of the list of all heads (Q's,
// then K's), the blockIdx.y-th `heads` of them.  Thread: one unit of one token,
// heads `lane`, lane + lanes, ... of those.
template <int MODE>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeTable t, const RopeArgs a)
{
    const int units = units_of(MODE, t.d, t.rot);
    const int slots = a.tile * units;
    const int lanes = kRopeThreads / slots;
    const int slot = threadIdx.x % slots, lane = threadIdx.x / slots;
    const int tiles = (a.s + a.tile - 1) / a.tile;
    const int batch = blockIdx.x / tiles;
    const int tok = (blockIdx.x % tiles) * a.tile + slot / units;
    if (lane >= lanes || tok >= a.s) return;
    const int64_t pos = a.positions ? a.positions[(int64_t)batch * a.s + tok] : (int64_t)a.pos0 + tok;
    Unit<MODE> un;
    un.place(t, slot % units);
    // Heads of Q, then of K, as one list.  The first ones' loads go out before the
    // angles are formed.
    const uint16_t* xq = a.q + batch * a.q_stride[0] + tok * a.q_stride[2];
    const uint16_t* xk = a.k + batch * a.k_stride[0] + tok * a.k_stride[2];
    uint16_t* yq = a.yq + batch * a.yq_stride[0] + tok * a.yq_stride[2];
    uint16_t* yk = a.yk + batch * a.yk_stride[0] + tok * a.yk_stride[2];
    const int h0 = (int)blockIdx.y * a.heads + lane;
    const int h1 = min(((int)blockIdx.y + 1) * a.heads, a.h_q + a.h_kv);
    auto load = [&](int h) {
        return un.load(h < a.h_q ? xq + h * a.q_stride[1] : xk + (h - a.h_q) * a.k_stride[1]);
    };
    auto store = [&](int h, const typename Unit<MODE>::Data& d) {
        un.store(h < a.h_q ? yq + h * a.yq_stride[1] : yk + (h - a.h_q) * a.yk_stride[1], d);
    };
    typename Unit<MODE>::Data d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i * lanes < h1) d[i] = load(h0 + i * lanes);
    un.turn(t, pos, a.sign);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i * lanes < h1) store(h0 + i * lanes, d[i]);
}

// One block: `tile` new tokens and a part of the heads, as rope_kernel's.
template <int MODE>
__global__ void __launch_bounds__(kRopeThreads) append_kernel(const __grid_constant__ RopeTable t, const AppendArgs a)
{
    const PagedTables& pt = a.t;
    const int units = units_of(MODE, t.d, t.rot);
    const int slots = a.tile * units;
    const int lanes = kRopeThreads / slots;
    const int slot = threadIdx.x % slots, lane = threadIdx.x / slots;
    const int tok0 = blockIdx.x * a.tile;
    const int tok = tok0 + slot / units;
    // the sequence of the tile's first token: the last one that starts at or before it
    int seq = -1;
    bool outside = false, falls = false;
    for (int i0 = 0; i0 <= pt.n_seq; i0 += kRopeThreads) {
        const int i = i0 + threadIdx.x;
        const bool here = i <= pt.n_seq;
        const int start = here ? pt.cu_q[i] : 0;
        if (here) outside |= start < 0 || start > pt.n_tokens;
        if (i < pt.n_seq) falls |= pt.cu_q[i + 1] < start;
        seq += __syncthreads_count(here && start <= tok0);
    }
    if ((outside || falls) && pt.status) atomicCAS(pt.status, 0, kStatusTable);
    // starts that decrease: which sequence owns a token (and the page row) is not known
    if (__syncthreads_or(falls)) return;
    if (lane >= lanes || tok >= pt.n_tokens) return;
    while (seq >= 0 && seq < pt.n_seq && pt.cu_q[seq + 1] <= tok) ++seq;
    if (seq < 0 || seq >= pt.n_seq) return;           // behind the last sequence: not ours
    const int q0 = pt.cu_q[seq], q1 = pt.cu_q[seq + 1], kv = pt.kv_lens[seq];
    if (q0 < 0 || q1 > pt.n_tokens) return;           // reported above
    const int64_t pos = (int64_t)kv - q1 + tok;
    int page = -1;
    if (pos >= 0 && kv <= (int64_t)pt.max_pages * pt.page_size)
        page = pt.page_table[(int64_t)seq * pt.max_pages + (pos >> pt.page_shift)];
    const bool placed = page >= 0 && page < pt.n_pages;
    if (!placed && pt.status) atomicCAS(pt.status, 0, kStatusTable);
    Unit<MODE> un;
    un.place(t, slot % units);
    // Heads of Q (where wanted), then of K, then of V, as one list; K's and V's go to
    // the page, if there is one for this token.
    const int d = t.d, h_q = a.q ? pt.h_q : 0;
    const int64_t row0 = ((int64_t)page * pt.h_kv * pt.page_size + (pos & (pt.page_size - 1))) * d;
    const int64_t head = (int64_t)pt.page_size * d;
    const int h0 = (int)blockIdx.y * a.heads + lane;
    const int all = h_q + (placed ? 2 * pt.h_kv : 0);
    const int h1 = min(((int)blockIdx.y + 1) * a.heads, all);
    auto load = [&](int h) {
        if (h < h_q) return un.load(a.q + tok * a.q_stride + h * d);
        h -= h_q;
        return un.load(h < pt.h_kv ? a.k + tok * a.k_stride + h * d : a.v + tok * a.v_stride + (h - pt.h_kv) * d);
    };
    auto store = [&](int h, const typename Unit<MODE>::Data& x) {
        if (h < h_q) {
            un.store(a.q_out + ((int64_t)tok * pt.h_q + h) * d, x);
        } else if (h - h_q < pt.h_kv) {
            un.store(a.k_pages + row0 + (h - h_q) * head, x);
        } else {
            un.store_raw(a.v_pages + row0 + (h - h_q - pt.h_kv) * head, x);
        }
    };
    typename Unit<MODE>::Data x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i * lanes < h1) x[i] = load(h0 + i * lanes);
    un.turn(t, pos, 1.0f);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i * lanes < h1) store(h0 + i * lanes, x[i]);
}

namespace {

int mode_of(const RopeTable& t) { return t.interleaved ? 2 : (t.rot % 16 == 0 ? 0 : 1); }

// Tokens per block: as many as fit its threads, so that each angle is formed once per
// block and a head's rows are read in long runs.  Heads per block: as many as a thread
// has loads in flight, so that all of its reads go out at once and none waits behind a
// write; fewer where that leaves an SM without eight blocks.  Measured on the
// [64 + 8, 8192, 128] layer and on [2, 12 + 12, 2048, 128] (half of each head), in a
// graph, with 2, 3, 4, 5, 6 and 8 heads and loads: 59.3 and 15.8 us, 48.7 and 13.0,
// 46.2 and 11.8, 46.6 and 11.3, 47.2 and 11.3, 47.1 and 11.9; two loads ahead in a
// longer loop: 48.4 to 49 and 13.3 to 14; 256 threads: 47.3 and 12.5.
constexpr int kBlocksPerSm = 8;
struct Split {
    int tile, heads;
    dim3 grid;
};
Split split(int units, int batches, int tokens, int heads, int sms)
{
    Split s;
    s.tile = 1;
    while (2 * s.tile * units <= kRopeThreads && s.tile < tokens) s.tile *= 2;
    const int lanes = kRopeThreads / (s.tile * units);
    const int64_t x = (int64_t)batches * ((tokens + s.tile - 1) / s.tile);
    int64_t groups = ((int64_t)kBlocksPerSm * sms + x - 1) / x;
    const int64_t by_heads = (heads + kAhead * lanes - 1) / (kAhead * lanes);
    groups = groups > by_heads ? groups : by_heads;
    groups = groups < heads ? groups : heads;
    s.heads = (int)((heads + groups - 1) / groups);
    s.grid = dim3((unsigned)x, (unsigned)((heads + s.heads - 1) / s.heads));
    return s;
}

}  // namespace

int launch_rope(const RopeTable& t, RopeArgs& a, int b, int sms, cudaStream_t st)
{
    const int mode = mode_of(t);
    const Split sp = split(units_of(mode, t.d, t.rot), b, a.s, a.h_q + a.h_kv, sms);
    a.tile = sp.tile;
    a.heads = sp.heads;
    const dim3 grid = sp.grid;
    if (mode == 0)
        rope_kernel<0><<<grid, kRopeThreads, 0, st>>>(t, a);
    else if (mode == 1)
        rope_kernel<1><<<grid, kRopeThreads, 0, st>>>(t, a);
    else
        rope_kernel<2><<<grid, kRopeThreads, 0, st>>>(t, a);
    return (int)cudaGetLastError();
}

int launch_append(const RopeTable& t, AppendArgs& a, int sms, cudaStream_t st)
{
    const int mode = mode_of(t);
    const Split sp = split(units_of(mode, t.d, t.rot), 1, a.t.n_tokens, (a.q ? a.t.h_q : 0) + 2 * a.t.h_kv, sms);
    a.tile = sp.tile;
    a.heads = sp.heads;
    const dim3 grid = sp.grid;
    if (mode == 0)
        append_kernel<0><<<grid, kRopeThreads, 0, st>>>(t, a);
    else if (mode == 1)
        append_kernel<1><<<grid, kRopeThreads, 0, st>>>(t, a);
    else
        append_kernel<2><<<grid, kRopeThreads, 0, st>>>(t, a);
    return (int)cudaGetLastError();
}

}  // namespace ac
