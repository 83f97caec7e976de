// prefix.cu -- attention over a paged cache of sequences that share their first pages.
//
// A group is a run of sequences whose page tables begin with the same pages.  Row r of
// its sequence i attends to the shared keys P and to the sequence's own S_i; with
//     (O_X, z_X) = softmax(scale q X^T) V over the keys X, and its log-sum-exp,
// O = (e^z_P O_P + e^z_S O_S) / (e^z_P + e^z_S) and LSE = ln(e^z_P + e^z_S).  So the
// shared keys are a sequence of their own, whose rows are all new tokens of the group
// and which hides no key from any of them: 128 rows of a tile visit a block of shared
// keys together, where the plain batch visits it once for each sequence.
//
// Three kernels, launched programmatically one behind the other:
//   plan   turns tables and groups into one list of sequences (PrefixSeq): the groups'
//          shared parts, then each sequence's own part
//   attend the kernel of paged_attn.cuh over that list; rows that have a part of their
//          softmax elsewhere leave as fp32 with their LSE
//   join   a warp per row adds its parts up
#include "paged_attn.cuh"

namespace ac {

namespace {

constexpr int kPlanThreads = 1024;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: rows [parts of cut tiles | whole tiles' rows, twice] of d floats, their
// base-2 LSEs, the records, the plan.
struct PrefixLayout {
    size_t lse, records, plan, bytes;
};
inline PrefixLayout prefix_layout(int d, int n_seq, int n_groups, int64_t n_tokens, int h_q, int h_kv)
{
    const size_t rows = (size_t)kPagedMaxCtas * 2 * 128 + 2 * (size_t)n_tokens * h_q;
    PrefixLayout l;
    l.lse = align256(rows * d * sizeof(float));
    l.records = align256(l.lse + rows * sizeof(float));
    l.plan = align256(l.records + 2 * (size_t)n_tokens * h_kv * sizeof(uint32_t));
    l.bytes = align256(l.plan + ((size_t)n_seq + n_groups) * sizeof(PrefixSeq));
    return l;
}

// Block 0 plans; all blocks clear the records of the sequences' own rows (a token that
// no tile covers must not find an earlier call's).  What a group shares in fact is what
// all its sequences hold before their first new token, in whole pages, so that no row's
// mask ends inside it; a group of one sequence shares nothing.  Groups out of order or
// out of range are reported and share nothing either: the attention is right without.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PagedTables t, int tpt, int causal,
                                                                   const PrefixGroups gr, PrefixSeq* plan,
                                                                   uint32_t* records, int n_records)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = (int)(blockIdx.x * blockDim.x + threadIdx.x); i < n_records; i += (int)(gridDim.x * blockDim.x))
        records[i] = kRecordNone;
    if (blockIdx.x) return;
    const int kind = causal ? 0 : kKindAll;
    for (int s = (int)threadIdx.x; s < t.n_seq; s += kPlanThreads) {
        const SeqTable q = read_seq(t, s, tpt, causal);
        if (q.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
        plan[gr.n + s] = PrefixSeq{q.q0, q.s.nq, q.s.kv, s, 0, kind, {}};
    }
    bool bad = false;
    for (int g = (int)threadIdx.x; g < gr.n; g += kPlanThreads)
        bad |= gr.starts[g] < 0 || gr.starts[g + 1] < gr.starts[g] || gr.starts[g + 1] > t.n_seq || gr.pages[g] < 0;
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
    const int lane = threadIdx.x & 31;
    for (int g = (int)(threadIdx.x >> 5); g < gr.n; g += kPlanThreads / 32) {
        PrefixSeq shared{};
        if (!bad) {
            const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
            int pages = gr.pages[g] < t.max_pages ? gr.pages[g] : t.max_pages;
            int members = 0, q0 = INT32_MAX, q1 = 0, row = INT32_MAX;
            for (int s = s0 + lane; s < s1; s += 32) {
                const SeqTable q = read_seq(t, s, tpt, causal);
                if (q.s.nq <= 0) continue;
                const int old = q.s.kv > q.s.nq ? (q.s.kv - q.s.nq) >> t.page_shift : 0;
                pages = old < pages ? old : pages;
                ++members;
                q0 = q.q0 < q0 ? q.q0 : q0;
                q1 = q.q0 + q.s.nq > q1 ? q.q0 + q.s.nq : q1;
                row = s < row ? s : row;
            }
            members = __reduce_add_sync(0xffffffffu, members);
            pages = __reduce_min_sync(0xffffffffu, pages);
            q0 = __reduce_min_sync(0xffffffffu, q0);
            q1 = __reduce_max_sync(0xffffffffu, q1);
            row = __reduce_min_sync(0xffffffffu, row);
            if (members > 1 && pages > 0) {
                shared = PrefixSeq{q0, q1 - q0, pages << t.page_shift, row, 0, kKindAll | kKindPrefix | kKindJoined, {}};
                for (int s = s0 + lane; s < s1; s += 32) {
                    const SeqTable q = read_seq(t, s, tpt, causal);
                    if (q.s.nq <= 0) continue;
                    plan[gr.n + s] = PrefixSeq{q.q0, q.s.nq, q.s.kv - (pages << t.page_shift), s, pages,
                                               kind | kKindJoined, {}};
                }
            }
        }
        if (lane == 0) plan[g] = shared;
    }
}

// A warp per (new token, query head): the parts of the row's own keys' tile, then of
// the group's.  As the join of cut tiles (paged.cu), with the rows found by records.
template <int D>
__global__ void __launch_bounds__(128) prefix_join_kernel(const PagedArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedTables& t = a.t;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)t.n_tokens * t.h_q) return;
    const int lane = threadIdx.x & 31;
    const int tok = (int)(row / t.h_q), head = (int)(row % t.h_q);
    const int kv_head = head / a.group, r_head = head % a.group;
    const uint32_t own = a.records[record_at(t, false, tok, kv_head)];
    if ((own & kRecordState) == kRecordNone) return;
    const uint32_t shared = own & kRecordJoined ? a.records[record_at(t, true, tok, kv_head)] : kRecordNone;
    auto count = [](uint32_t r) -> int {
        const uint32_t state = r & kRecordState;
        return state == kRecordNone ? 0 : state == kRecordWhole ? 1 : (int)((r >> 18 & 255) - (r >> 10 & 255)) + 1;
    };
    const int n_own = count(own), parts = n_own + count(shared);
    auto row_of = [&](int p) -> size_t {
        const bool prefix = p >= n_own;
        const uint32_t r = prefix ? shared : own;
        const int i = prefix ? p - n_own : p;
        if ((r & kRecordState) == kRecordWhole) return whole_row(t, prefix, tok, head);
        return part_row((int)(r >> 10 & 255) + i, i == 0 ? 1 : 0) + (r >> 3 & 127) + r_head;
    };
    const float* lse = reinterpret_cast<const float*>(a.ws + a.lse_offset);
    const float* rows = reinterpret_cast<const float*>(a.ws) + lane;
    constexpr int E = D / 32, AHEAD = 4;
    float x[AHEAD][E];
    auto load = [&](int p0) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (p0 + k < parts) {
                const float* from = rows + row_of(p0 + k) * D;
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] = from[e * 32];
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
    uint16_t* orow = a.o + (size_t)row * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e * 32] = (uint16_t)(pack_bf16x2(acc[e] * inv, 0.f) & 0xffffu);
    if (lane == 0)
        a.lse[(size_t)head * t.n_tokens + tok] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945309f;
}

template <typename... Args>
cudaError_t launch_behind(void (*kern)(Args...), dim3 grid, int threads, uint32_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
int launch_prefix_t(const PagedMaps& m, PagedArgs a, const PrefixGroups& g, cudaStream_t st)
{
    const PagedTables& t = a.t;
    const PrefixLayout l = prefix_layout(D, t.n_seq, g.n, t.n_tokens, t.h_q, t.h_kv);
    PrefixSeq* plan = reinterpret_cast<PrefixSeq*>(a.ws + l.plan);
    a.plan = plan;
    a.n_plan = g.n + t.n_seq;
    a.records = reinterpret_cast<uint32_t*>(a.ws + l.records);
    a.lse_offset = l.lse;
    const int n_records = t.n_tokens * t.h_kv;
    const int clearing = n_records / (kPlanThreads * 8);
    prefix_plan_kernel<<<(unsigned)(clearing < 1 ? 1 : clearing < 64 ? clearing : 64), kPlanThreads, 0, st>>>(
        t, a.tpt, a.causal, g, plan, a.records, n_records);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;

    constexpr uint32_t smem = PagedCfg<D>::SMEM;
    const bool fine = (int64_t)t.n_tokens * a.group <= (int64_t)kFineRows * t.n_seq;      // as launch_paged_t
    auto kern = fine ? paged_attn_kernel<D, true, true> : paged_attn_kernel<D, false, true>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return (int)e;
    const int64_t blocks = ((int64_t)t.max_pages * t.page_size + 127) / 128;
    const int64_t row_tiles = ((int64_t)t.n_tokens + a.tpt - 1) / a.tpt;
    const int64_t want = ((2 * row_tiles + a.n_plan) * t.h_kv * blocks + kMinUnits - 1) / kMinUnits;
    int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
    if (want < grid) grid = want;
    if ((e = launch_behind(kern, dim3((unsigned)grid), kThreads, smem, st, m, a)) != cudaSuccess) return (int)e;
    const int64_t rows = (int64_t)t.n_tokens * t.h_q;
    return (int)launch_behind(prefix_join_kernel<D>, dim3((unsigned)((rows + 3) / 4)), 128, 0, st, a);
}

}  // namespace

size_t prefix_ws_bytes(int d, int n_seq, int n_groups, int64_t n_tokens, int h_q, int h_kv)
{
    return prefix_layout(d, n_seq, n_groups, n_tokens, h_q, h_kv).bytes;
}

int launch_prefix(const PagedMaps& m, const PagedArgs& a, const PrefixGroups& g, cudaStream_t st)
{
    switch (a.d) {
        case 64: return launch_prefix_t<64>(m, a, g, st);
        case 96: return launch_prefix_t<96>(m, a, g, st);
        case 128: return launch_prefix_t<128>(m, a, g, st);
        case 160: return launch_prefix_t<160>(m, a, g, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
