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
// sines in registers and walks over the heads, so the angles cost one
// evaluation per (token, unit, head lane) and no shared memory.
#include "kernels.h"
#include "ptx.cuh"

namespace ac {

namespace {

constexpr int kRopeThreads = 256;

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

    __device__ __forceinline__ void init(const RopeTable& t, int unit, int64_t pos, float sign)
    {
        u = unit;
        rot = t.rot;
        half = t.rot / 2;
        n_pair_units = half / PAIRS;
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

// One block: `tile` tokens of one batch element, all heads.  Thread: one unit of
// one token, heads `lane`, lane + n_lanes, ...
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
    un.init(t, slot % units, pos, a.sign);
    auto walk = [&](const uint16_t* x, const int64_t (&xs)[3], uint16_t* y, const int64_t (&ys)[3], int heads,
                    int first) {
        const uint16_t* xr = x + batch * xs[0] + tok * xs[2];
        uint16_t* yr = y + batch * ys[0] + tok * ys[2];
        for (int h = first; h < heads; h += 2 * lanes) {
            const bool two = h + lanes < heads;
            const auto d0 = un.load(xr + h * xs[1]);
            const auto d1 = two ? un.load(xr + (h + lanes) * xs[1]) : d0;
            un.store(yr + h * ys[1], d0);
            if (two) un.store(yr + (h + lanes) * ys[1], d1);
        }
    };
    walk(a.q, a.q_stride, a.yq, a.yq_stride, a.h_q, lane);
    walk(a.k, a.k_stride, a.yk, a.yk_stride, a.h_kv, lane);
}

// One block: `tile` new tokens, all heads of Q, K and V.
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
    for (int i0 = 0; i0 <= pt.n_seq; i0 += kRopeThreads) {
        const int i = i0 + threadIdx.x;
        seq += __syncthreads_count(i <= pt.n_seq && pt.cu_q[i] <= tok0);
    }
    if (lane >= lanes || tok >= pt.n_tokens) return;
    while (seq >= 0 && seq < pt.n_seq && pt.cu_q[seq + 1] <= tok) ++seq;
    if (seq < 0 || seq >= pt.n_seq) return;           // behind the last sequence: not ours
    const int q0 = pt.cu_q[seq], q1 = pt.cu_q[seq + 1], kv = pt.kv_lens[seq];
    if (q0 < 0 || tok < q0 || q1 > pt.n_tokens) {     // not a table of increasing starts
        if (pt.status) atomicCAS(pt.status, 0, kStatusTable);
        return;
    }
    const int64_t pos = (int64_t)kv - q1 + tok;
    int page = -1;
    if (pos >= 0 && kv <= (int64_t)pt.max_pages * pt.page_size)
        page = pt.page_table[(int64_t)seq * pt.max_pages + (pos >> pt.page_shift)];
    const bool placed = page >= 0 && page < pt.n_pages;
    if (!placed && pt.status) atomicCAS(pt.status, 0, kStatusTable);
    Unit<MODE> un;
    un.init(t, slot % units, pos, 1.0f);
    const int d = t.d;
    if (a.q) {
        const uint16_t* x = a.q + tok * a.q_stride;
        uint16_t* y = a.q_out + (int64_t)tok * pt.h_q * d;
        for (int h = lane; h < pt.h_q; h += 2 * lanes) {
            const bool two = h + lanes < pt.h_q;
            const auto d0 = un.load(x + h * d);
            const auto d1 = two ? un.load(x + (h + lanes) * d) : d0;
            un.store(y + h * d, d0);
            if (two) un.store(y + (h + lanes) * d, d1);
        }
    }
    if (!placed) return;
    const int64_t row0 = ((int64_t)page * pt.h_kv * pt.page_size + (pos & (pt.page_size - 1))) * d;
    const int64_t head = (int64_t)pt.page_size * d;
    for (int h = lane; h < pt.h_kv; h += lanes) {
        const auto dk = un.load(a.k + tok * a.k_stride + h * d);
        const auto dv = un.load(a.v + tok * a.v_stride + h * d);
        un.store(a.k_pages + row0 + h * head, dk);
        un.store_raw(a.v_pages + row0 + h * head, dv);
    }
}

namespace {

int mode_of(const RopeTable& t) { return t.interleaved ? 2 : (t.rot % 16 == 0 ? 0 : 1); }

// Tokens per block: as many as fit the block's threads (fewer evaluations of each
// angle), but no more than leaves four blocks for every SM, so that short calls
// spread over the whole chip.
int tile_of(int units, int64_t tokens, int sms)
{
    int tile = 1;
    while (2 * tile * units <= kRopeThreads && tokens / (2 * tile) >= 4ll * sms) tile *= 2;
    return tile;
}

}  // namespace

int launch_rope(const RopeTable& t, RopeArgs& a, int b, int sms, cudaStream_t st)
{
    const int mode = mode_of(t);
    a.tile = tile_of(units_of(mode, t.d, t.rot), (int64_t)b * a.s, sms);
    const unsigned grid = (unsigned)b * (unsigned)((a.s + a.tile - 1) / a.tile);
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
    a.tile = tile_of(units_of(mode, t.d, t.rot), a.t.n_tokens, sms);
    const unsigned grid = (unsigned)((a.t.n_tokens + a.tile - 1) / a.tile);
    if (mode == 0)
        append_kernel<0><<<grid, kRopeThreads, 0, st>>>(t, a);
    else if (mode == 1)
        append_kernel<1><<<grid, kRopeThreads, 0, st>>>(t, a);
    else
        append_kernel<2><<<grid, kRopeThreads, 0, st>>>(t, a);
    return (int)cudaGetLastError();
}

}  // namespace ac
