// paged.cu -- attention of new tokens over a paged key/value cache: the join of cut
// tiles' parts, and the launches (the attention kernel is in paged_attn.cuh).
#include "paged_attn.cuh"

namespace ac {

// Joins the parts of the tiles that were cut: block (c, y) takes rows 4y .. 4y + 3 of
// the tile that CTA c cut at its end, a warp per row.  Up to 32 parts at a time: lane
// p forms part p's weight, then lanes over d sum the parts' rows, eight in flight and
// the first eight on their way while the weights are formed (a chain of loads is all
// that this kernel's time consists of).  Launched programmatically, it waits for the
// attention kernel's end.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedTables& t = a.t;
    const CutTile cut = reinterpret_cast<const CutTile*>(a.ws + ws_cut_offset(D))[blockIdx.x];
    const int lane = threadIdx.x & 31;
    const int r = (int)blockIdx.y * 4 + (int)(threadIdx.x >> 5);
    if (cut.last_cta == 0 || r >= cut.n_rows) return;
    const int parts = cut.last_cta - (int)blockIdx.x + 1;
    const float* lse = reinterpret_cast<const float*>(a.ws + ws_lse_offset(D));
    const float* rows = reinterpret_cast<const float*>(a.ws) + lane;
    auto row_of = [&](int p) { return part_row((int)blockIdx.x + p, p == 0 ? 1 : 0) + r; };
    constexpr int E = D / 32, AHEAD = 8;
    float x[AHEAD][E];
    auto load = [&](int p0) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (p0 + k < parts) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] = rows[row_of(p0 + k) * D + e * 32];
            }
    };
    float m = -INFINITY, sum = 0.f, acc[E] = {};
    for (int p0 = 0; p0 < parts; p0 += 32) {
        const float z = p0 + lane < parts ? lse[row_of(p0 + lane)] : -INFINITY;
        load(p0);
        float top = z;
#pragma unroll
        for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m_new = fmaxf(m, top);
        const float m_ref = m_new == -INFINITY ? 0.f : m_new;
        const float f = exp2f(m - m_ref);                     // 0 the first time
        const float w = exp2f(z - m_ref);
        m = m_new;
        float ws = w;
#pragma unroll
        for (int o = 16; o; o /= 2) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        sum = sum * f + ws;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
        for (int p = p0; p < parts && p < p0 + 32; p += AHEAD) {
            if (p > p0) load(p);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, (p - p0 + k) & 31);
                if (p + k < parts) {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += wk * x[k][e];
                }
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;       // NaN stays
    const int tok = cut.q_tok + r / a.group, head = cut.head * a.group + r % a.group;
    uint16_t* orow = a.o + ((size_t)tok * t.h_q + head) * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e * 32] = (uint16_t)(pack_bf16x2(acc[e] * inv, 0.f) & 0xffffu);
    if (lane == 0)
        a.lse[(size_t)head * t.n_tokens + tok] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945309f;
}

size_t paged_ws_bytes(int d) { return ws_counter_offset(d) + 256; }

int paged_tokens_per_tile(int group) { return 128 / group; }

namespace {

template <int D>
int launch_paged_t(const PagedMaps& m, const PagedArgs& args, cudaStream_t st)
{
    constexpr uint32_t smem = PagedCfg<D>::SMEM;
    // new tokens that make tiles of few rows, on average
    auto kern = fine_batch(args) ? paged_attn_kernel<D, true, false> : paged_attn_kernel<D, false, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
    // The most units that the tables can ask for bounds the grid (short batches
    // need few CTAs), and the most blocks of a tile tells whether any can be cut.
    const int64_t blocks = ((int64_t)args.t.max_pages * args.t.page_size + 127) / 128;
    const int64_t tiles = (((int64_t)args.t.n_tokens + args.tpt - 1) / args.tpt + args.t.n_seq) * args.t.h_kv;
    const int64_t want = (tiles * blocks + kMinUnits - 1) / kMinUnits;
    PagedArgs a = args;
    int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
    if (want < grid) grid = want;
    // The kernel may hand out tiles where hand_out_tiles() could say so of any lengths
    // that these sizes allow, tiles may be longer than the 8 blocks up to which many stay
    // whole anyway (272 tiles of 5 blocks: 28 us so), and sequences have half a tile's new
    // tokens on average, not one or two.  The counter starts at 0; setting it costs 3 to
    // 7 us, so other batches do without.
    const int64_t least = ((int64_t)a.t.n_tokens + a.tpt - 1) / a.tpt * a.t.h_kv;         // tiles
    const int64_t most_bytes = (int64_t)a.t.n_seq * a.t.max_pages * a.t.page_size * a.t.h_kv * (4 * D);
    if (blocks > 8 && 10 * tiles >= 14 * grid && 2ll * a.t.n_tokens >= (int64_t)a.tpt * a.t.n_seq &&
        a.t.n_tokens >= 2ll * a.t.n_seq && (2 * least <= 5 * grid || most_bytes > kManyBytes)) {
        a.counter = reinterpret_cast<uint32_t*>(a.ws + ws_counter_offset(D));
        if ((e = cudaMemsetAsync(a.counter, 0, sizeof(uint32_t), st)) != cudaSuccess) return (int)e;
    }
    kern<<<(unsigned)grid, kThreads, smem, st>>>(m, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return (int)e;
    if (grid > 1 && blocks > kLeastSnap) {
        const int64_t rows = (int64_t)(a.tpt < a.t.n_tokens ? a.tpt : a.t.n_tokens) * a.group;
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)grid, (unsigned)((rows + 3) / 4));
        cfg.blockDim = dim3(128);
        cfg.stream = st;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a);
    }
    return (int)e;
}

}  // namespace

int launch_paged(const PagedMaps& m, const PagedArgs& a, cudaStream_t st)
{
    switch (a.d) {
        case 64: return launch_paged_t<64>(m, a, st);
        case 96: return launch_paged_t<96>(m, a, st);
        case 128: return launch_paged_t<128>(m, a, st);
        case 160: return launch_paged_t<160>(m, a, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
