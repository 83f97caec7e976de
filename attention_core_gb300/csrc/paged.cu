// paged.cu -- attention of new tokens over a paged key/value cache on sm_103a.
//
// O = softmax(scale q K^T + mask) V and LSE, per (new token, query head).
// One warp per row: lanes take a key each for the scores and a slice of d for
// the sums, 32 keys at a time, with a running maximum and sum in fp32.
#include "kernels.h"
#include "ptx.cuh"

namespace ac {

template <int D>
__global__ void __launch_bounds__(128) paged_simple_kernel(const PagedArgs a)
{
    const PagedTables& t = a.t;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)t.n_tokens * t.h_q) return;
    const int tok = (int)(row / t.h_q), head = (int)(row % t.h_q);
    int seq = 0;
    while (seq < t.n_seq && t.cu_q[seq + 1] <= tok) ++seq;
    if (seq >= t.n_seq) return;
    const int q0 = t.cu_q[seq], q1 = t.cu_q[seq + 1], kv = t.kv_lens[seq];
    if (q0 < 0 || tok < q0 || q1 > t.n_tokens || kv < 0 || kv > (int64_t)t.max_pages * t.page_size) {
        if (t.status) atomicCAS(t.status, 0, kStatusTable);
        return;
    }
    const int64_t seen64 = a.causal ? (int64_t)kv - q1 + tok + 1 : kv;
    const int seen = (int)(seen64 < 0 ? 0 : seen64);
    for (int c = lane; c < D; c += 32) qs[warp][c] = __uint_as_float((uint32_t)a.q[row * D + c] << 16);
    __syncwarp();
    const int hk = head / (t.h_q / t.h_kv);
    float m = -INFINITY, l = 0.f, acc[D / 32] = {};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        int64_t base = 0;
        float x = -INFINITY;
        if (j < seen) {
            const int page = t.page_table[(int64_t)seq * t.max_pages + (j >> t.page_shift)];
            if (page < 0 || page >= t.n_pages) {
                if (t.status) atomicCAS(t.status, 0, kStatusTable);
            } else {
                base = (((int64_t)page * t.h_kv + hk) * t.page_size + (j & (t.page_size - 1))) * D;
            }
            float dot = 0.f;
            for (int c = 0; c < D; ++c) dot += qs[warp][c] * __uint_as_float((uint32_t)a.k_pages[base + c] << 16);
            x = dot * a.scale_log2;
        }
        float mx = x;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m, mx);
        const float f = exp2f(m - m_new);
        const float p = exp2f(x - m_new);
        l *= f;
        for (int e = 0; e < D / 32; ++e) acc[e] *= f;
        float ps = p;
        for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l += ps;
        m = m_new;
        for (int i = 0; i < 32 && j0 + i < seen; ++i) {
            const float pi = __shfl_sync(0xffffffffu, p, i);
            const int64_t bi = __shfl_sync(0xffffffffu, base, i);
            for (int e = 0; e < D / 32; ++e)
                acc[e] += pi * __uint_as_float((uint32_t)a.v_pages[bi + e * 32 + lane] << 16);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < D / 32; ++e)
        a.o[row * D + e * 32 + lane] = (uint16_t)(pack_bf16x2(acc[e] * inv, 0.f) & 0xffffu);
    if (lane == 0)
        a.lse[(int64_t)head * t.n_tokens + tok] = l > 0.f ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

size_t paged_ws_bytes(int) { return 256; }

int launch_paged(const PagedArgs& a, cudaStream_t st)
{
    const unsigned grid = (unsigned)(((int64_t)a.t.n_tokens * a.t.h_q + 3) / 4);
    switch (a.d) {
        case 64: paged_simple_kernel<64><<<grid, 128, 0, st>>>(a); break;
        case 96: paged_simple_kernel<96><<<grid, 128, 0, st>>>(a); break;
        case 128: paged_simple_kernel<128><<<grid, 128, 0, st>>>(a); break;
        case 160: paged_simple_kernel<160><<<grid, 128, 0, st>>>(a); break;
        default: return (int)cudaErrorInvalidValue;
    }
    return (int)cudaGetLastError();
}

}  // namespace ac
