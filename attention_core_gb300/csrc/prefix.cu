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
// Four kernels, launched programmatically one behind the other:
//   plan   turns tables and groups into one list of sequences (PrefixSeq): the groups'
//          shared parts, then each sequence's own part
//   attend the kernel of paged_attn.cuh over the list's sequences of many rows; rows that
//          have a part of their softmax elsewhere leave as fp32 with their LSE
//   few    the sequences of few rows (a sample's own keys, its single token)
//   join   a warp per row adds its parts up
#include "paged_attn.cuh"

namespace ac {

namespace {

constexpr int kPlanThreads = 1024;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: rows [parts of cut tiles | whole tiles' rows, twice | parts of cut tiles of
// few rows] of d floats, their base-2 LSEs, the records, the plan.
constexpr int kFewWarps = kPagedMaxCtas * 8;      // of the kernel for few rows, at most
struct PrefixLayout {
    size_t lse, records, plan, many, bytes;
};
__host__ __device__ inline size_t few_row(const PagedTables& t, int warp, int slot)
{
    return (size_t)kPagedMaxCtas * 2 * 128 + 2 * (size_t)t.n_tokens * t.h_q + ((size_t)warp * 2 + slot) * 16;
}
inline PrefixLayout prefix_layout(int d, int n_seq, int n_groups, int64_t n_tokens, int h_q, int h_kv)
{
    const size_t rows = (size_t)kPagedMaxCtas * 2 * 128 + 2 * (size_t)n_tokens * h_q + (size_t)kFewWarps * 2 * 16;
    PrefixLayout l;
    l.lse = align256(rows * d * sizeof(float));
    l.records = align256(l.lse + rows * sizeof(float));
    l.plan = align256(l.records + 2 * (size_t)n_tokens * h_kv * sizeof(uint64_t));
    l.many = align256(l.plan + ((size_t)n_seq + n_groups) * sizeof(PrefixSeq));
    l.bytes = l.many + 256;
    return l;
}

// Sequences of few rows: at most two tiles of 16 rows (16 / group tokens each).
constexpr int kFewKeys = 64;
__host__ __device__ inline bool few_rows(int nq, int group) { return nq > 0 && group <= 16 && nq <= 2 * (16 / group); }
__host__ __device__ inline int few_tiles(int nq, int group) { return (nq + 16 / group - 1) / (16 / group); }
__host__ __device__ inline int few_blocks(int kv) { return kv > 0 ? (int)(((uint32_t)kv + kFewKeys - 1) / kFewKeys) : 1; }

// Block 0 plans; all blocks clear the records of the sequences' own rows (a token that
// no tile covers must not find an earlier call's).  What a group shares in fact is what
// all its sequences hold before their first new token, in whole pages, so that no row's
// mask ends inside it; a group of one sequence shares nothing.  Groups out of order or
// out of range are reported and share nothing either: the attention is right without.
// The sequences' lengths are read once and kept in shared memory (the first kPlanNear of
// them: all, in any usual batch), since this kernel's time is what the others wait for.
constexpr int kPlanNear = 1024;
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PagedTables t, int tpt, int causal,
                                                                   const PrefixGroups gr, PrefixSeq* plan,
                                                                   uint64_t* records, int n_records,
                                                                   int64_t* many_units)
{
    __shared__ int4 near[kPlanNear];                 // first token, new tokens, keys, shared pages of a sequence
    __shared__ int64_t warp_units[kPlanThreads / 32];
    __shared__ unsigned long long many;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int g = tid; g < gr.n; g += kPlanThreads) {
            const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
            bad |= s0 < 0 || s1 < s0 || s1 > t.n_seq || gr.pages[g] < 0;
        }
        for (int s = tid; s < t.n_seq && s < kPlanNear; s += kPlanThreads) {
            const SeqTable q = read_seq(t, s, tpt, causal);
            if (q.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
            near[s] = make_int4(q.q0, q.s.nq, q.s.kv, 0);
        }
        if (tid == 0) many = 0;
        auto seq = [&](int s) -> int4 {
            if (s < kPlanNear) return near[s];
            const SeqTable q = read_seq(t, s, tpt, causal);
            if (q.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
            return make_int4(q.q0, q.s.nq, q.s.kv, 0);
        };
        // (beyond kPlanNear the shared pages go by way of the plan itself)
        for (int s = kPlanNear + tid; s < t.n_seq; s += kPlanThreads) plan[gr.n + s].page0 = 0;
        bad = __syncthreads_or(bad);
        if (bad && tid == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
        for (int g = warp; g < gr.n; g += kPlanThreads / 32) {
            PrefixSeq shared{};
            if (!bad) {
                const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
                int pages = gr.pages[g] < t.max_pages ? gr.pages[g] : t.max_pages;
                int members = 0, q0 = INT32_MAX, q1 = 0, row = INT32_MAX;
                for (int s = s0 + lane; s < s1; s += 32) {
                    const int4 q = seq(s);
                    if (q.y <= 0) continue;
                    const int old = q.z > q.y ? (q.z - q.y) >> t.page_shift : 0;
                    pages = old < pages ? old : pages;
                    ++members;
                    q0 = q.x < q0 ? q.x : q0;
                    q1 = q.x + q.y > q1 ? q.x + q.y : q1;
                    row = s < row ? s : row;
                }
                members = __reduce_add_sync(0xffffffffu, members);
                pages = __reduce_min_sync(0xffffffffu, pages);
                q0 = __reduce_min_sync(0xffffffffu, q0);
                q1 = __reduce_max_sync(0xffffffffu, q1);
                row = __reduce_min_sync(0xffffffffu, row);
                if (members > 1 && pages > 0) {
                    shared = PrefixSeq{q0, q1 - q0, pages << t.page_shift, row, 0, kKindAll | kKindPrefix | kKindJoined, 0};
                    for (int s = s0 + lane; s < s1; s += 32) {
                        if (s < kPlanNear)
                            near[s].w = pages;
                        else
                            plan[gr.n + s].page0 = pages;
                    }
                }
            }
            if (lane == 0) plan[g] = shared;
        }
        __syncthreads();
        // each sequence's own part, who has it, and the line of the kernel for few rows
        const int group = t.h_q / t.h_kv, n = gr.n + t.n_seq;
        int64_t base = 0;
        for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
            const int i = i0 + tid, s = i - gr.n;
            int64_t units = 0;
            PrefixSeq v{};
            if (i < n) {
                if (s < 0) {
                    v = plan[i];
                } else {
                    const int4 q = seq(s);
                    const int pages = q.y <= 0 ? 0 : s < kPlanNear ? q.w : plan[i].page0;
                    v = PrefixSeq{q.x, q.y, q.z - (pages << t.page_shift), s, pages,
                                  (causal ? 0 : kKindAll) | (pages ? kKindJoined : 0), 0};
                }
                if (few_rows(v.nq, group)) {
                    v.kind |= kKindFew;
                    units = (int64_t)few_tiles(v.nq, group) * few_blocks(v.kv) * t.h_kv;
                } else if (v.nq > 0) {
                    const SeqShape q{v.nq, v.kv, tpt, !(v.kind & kKindAll)};
                    atomicAdd(&many, (unsigned long long)q.units(q.tiles()) * t.h_kv);
                }
            }
            int64_t upto = units;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            if (lane == 31) warp_units[warp] = upto;
            __syncthreads();
            int64_t before = 0, all = 0;
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                const int64_t x = warp_units[w];
                if (w < warp) before += x;
                all += x;
            }
            if (i < n) {
                v.few_units = base + before + upto;
                plan[i] = v;
            }
            base += all;
            __syncthreads();
        }
        if (tid == 0) *many_units = (int64_t)many;
    }
    for (int i = (int)(blockIdx.x * blockDim.x) + tid; i < n_records; i += (int)(gridDim.x * blockDim.x))
        records[i] = kRecordNone;
}

// Attention of sequences of few rows (at most two tiles of 16) over their keys.  A tile
// of 128 rows takes several microseconds from its Q to its O however few of them are used,
// one after another on a processor: 64 samples' own 250 keys took 60 us that way.  Here a
// warp has a tile's piece by itself, eight on a processor, each with its own ring of
// 16-key steps of K and V (cp.async; 8 KB a step, so that about 100 KB are on their way to
// a processor) and its own softmax: S = Q K^T and O += P V by mma.m16n8k16, whose scores'
// layout is the layout that P needs.  Bound by the keys' bytes.  P goes in as two bf16
// terms, as in paged_attn.cuh's tiles of few rows.
// The units are blocks of 64 keys of (sequence, KV head, row tile), in equal shares for
// all warps; pieces of a tile are joined.  The kernel runs beside the one for many rows:
// that one keeps to as many processors as its part of the work is worth (many_ctas), and
// this one's blocks of lowest number, which are placed first, find the others free.
template <int D>
struct FewCfg {
    static constexpr int UNITS = D / 8;                        // of 16 bytes a row
    static constexpr uint32_t PITCH = (UNITS + 1) * 16;        // odd in 16 bytes: ldmatrix meets no bank twice
    static constexpr uint32_t TILE = 16 * PITCH, STAGE = 2 * TILE;
    static constexpr int STAGES = D <= 96 ? 4 : 3;
    static constexpr int WARPS = D <= 128 ? 8 : 7;
    static constexpr uint32_t SMEM = WARPS * STAGES * STAGE;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// The plan was written before this kernel began, but it waits for no kernel before it
// reads: past L1.
__device__ __forceinline__ PrefixSeq load_plan(const PrefixSeq* p)
{
    static_assert(sizeof(PrefixSeq) == 32, "two loads");
    union {
        int4 x[2];
        PrefixSeq v;
    } u;
    u.x[0] = __ldcg(reinterpret_cast<const int4*>(p));
    u.x[1] = __ldcg(reinterpret_cast<const int4*>(p) + 1);
    return u.v;
}

struct FewSegment {
    PrefixSeq v;
    int head, q_tok, n_tok;
    int first_pos;          // position of the tile's first token among the sequence's keys
    int k0, k1;             // keys [k0, k1)
    bool whole, from_start;
    int last;               // of a cut tile's first piece: the warp of its last one
};

struct FewWalk {
    int64_t at, end, per;
    int s, head, m, b;
    PrefixSeq v;

    // Unit u0 is in the first of the sequences lo .. hi - 1 whose units reach beyond it.
    __device__ __forceinline__ void start(const PrefixSeq* plan, int lo, int hi, int h_kv, int group, int64_t u0, int64_t u1)
    {
        at = u0;
        end = u1;
        const int lane = threadIdx.x & 31;
        while (hi - lo > 32) {                             // 32 candidates a round
            const int step = (hi - lo + 31) / 32;
            const int last = lo + (lane + 1) * step - 1 < hi ? lo + (lane + 1) * step - 1 : hi - 1;
            const uint32_t beyond = __ballot_sync(0xffffffffu, __ldcg(&plan[last].few_units) > u0);
            lo += (__ffs(beyond) - 1) * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        const PrefixSeq c = load_plan(plan + (lo + lane < hi ? lo + lane : hi - 1));
        const int src = __ffs(__ballot_sync(0xffffffffu, c.few_units > u0)) - 1;
        s = lo + src;
        v.q0 = __shfl_sync(0xffffffffu, c.q0, src);
        v.nq = __shfl_sync(0xffffffffu, c.nq, src);
        v.kv = __shfl_sync(0xffffffffu, c.kv, src);
        v.row = __shfl_sync(0xffffffffu, c.row, src);
        v.page0 = __shfl_sync(0xffffffffu, c.page0, src);
        v.kind = __shfl_sync(0xffffffffu, c.kind, src);
        v.few_units = __shfl_sync(0xffffffffu, c.few_units, src);
        const int blocks = few_blocks(v.kv), per_head = few_tiles(v.nq, group) * blocks;
        const int64_t rel = u0 - (v.few_units - (int64_t)per_head * h_kv);
        head = (int)quot(rel, per_head);
        const int in_head = (int)(rel - (int64_t)head * per_head);
        m = in_head / blocks;
        b = in_head - m * blocks;
    }

    __device__ __forceinline__ bool next(const PrefixSeq* plan, int n_plan, int h_kv, int group, FewSegment& g)
    {
        if (at >= end) return false;
        int blocks = few_blocks(v.kv);
        if (b >= blocks) {
            b = 0;
            if (++m >= few_tiles(v.nq, group)) {
                m = 0;
                if (++head >= h_kv) {
                    head = 0;
                    do {
                        if (++s >= n_plan) {               // only past the line's end
                            at = end;
                            return false;
                        }
                        v = load_plan(plan + s);
                    } while (!(v.kind & kKindFew));
                    blocks = few_blocks(v.kv);
                }
            }
        }
        const int take = end - at < blocks - b ? (int)(end - at) : blocks - b;
        const int tpt = 16 / group;
        g.v = v;
        g.head = head;
        g.q_tok = v.q0 + m * tpt;
        g.n_tok = v.nq - m * tpt < tpt ? v.nq - m * tpt : tpt;
        g.first_pos = v.kv - v.nq + m * tpt;
        g.k0 = b * kFewKeys;
        g.k1 = (b + take) * kFewKeys < v.kv ? (b + take) * kFewKeys : v.kv;
        g.whole = take == blocks;
        g.from_start = b == 0;
        g.last = g.whole || !g.from_start ? 0 : (int)quot(at + (blocks - b) - 1, per);
        at += take;
        b += take;
        return true;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// D [16 x 8] += A [16 x 16] B [16 x 8], bf16 in, fp32 sums
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(FewCfg<D>::WARPS * 32, 1)
prefix_few_kernel(const PagedArgs a, const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages)
{
    using C = FewCfg<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const PagedTables& t = a.t;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.group;
    const uint32_t ring = smem_u32(smem_raw) + warp * C::STAGES * C::STAGE;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.few_waits) asm volatile("griddepcontrol.wait;" ::: "memory");

    // The line's length, and 32 places of it in the same look: this warp's share starts
    // between two of them.
    const int step = (a.n_plan + 31) / 32;
    const int last = (lane + 1) * step < a.n_plan ? (lane + 1) * step - 1 : a.n_plan - 1;
    const int64_t upto = __ldcg(&a.plan[last].few_units), many = __ldcg(a.many_units);
    const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
    const int blocks = (int)gridDim.x - (many > 0 ? (int)many_ctas(many, total, gridDim.x) : 0);
    const int n_blocks = blocks > 0 ? blocks : 1;
    const int me = warp * n_blocks + (int)blockIdx.x;      // neighbouring shares on different processors
    int64_t per = quot(total + (int64_t)n_blocks * C::WARPS - 1, (int64_t)n_blocks * C::WARPS);
    per = per > 1 ? per : 1;
    const int64_t u0 = me * per, u1 = u0 + per < total ? u0 + per : total;
    if ((int)blockIdx.x >= n_blocks || u0 >= u1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int lo = (__ffs(__ballot_sync(0xffffffffu, upto > u0)) - 1) * step;
    FewWalk load_walk;
    load_walk.per = per;
    load_walk.start(a.plan, lo, lo + step < a.n_plan ? lo + step : a.n_plan, t.h_kv, group, u0, u1);
    FewWalk walk = load_walk;

    // ---- loads: 16 keys a step, the entries of the page table 32 at a time
    FewSegment lg;
    int lk = 0, window = 0, entry = -1;
    bool loading = load_walk.next(a.plan, a.n_plan, t.h_kv, group, lg);
    auto fetch_entries = [&](int first) {
        window = first;
        const int i = first + lane, n = (lg.v.kv + t.page_size - 1) >> t.page_shift;
        entry = i < n ? t.page_table[(int64_t)lg.v.row * t.max_pages + lg.v.page0 + i] : -1;
    };
    if (loading) {
        lk = lg.k0;
        fetch_entries(lk >> t.page_shift);
    }
    int load_slot = 0;
    auto issue = [&]() {
        while (loading && lk >= lg.k1) {
            loading = load_walk.next(a.plan, a.n_plan, t.h_kv, group, lg);
            if (loading) {
                lk = lg.k0;
                fetch_entries(lk >> t.page_shift);
            }
        }
        if (loading) {
            if ((lk >> t.page_shift) >= window + 32) fetch_entries(lk >> t.page_shift);
            const int page = __shfl_sync(0xffffffffu, entry, (lk >> t.page_shift) - window);
            const bool there = page >= 0 && page < t.n_pages;
            if (!there && lane == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
            const size_t row0 = there ? ((size_t)page * t.h_kv + lg.head) * t.page_size + (lk & (t.page_size - 1)) : 0;
            const int rows = there ? lg.k1 - lk : 0;           // what lies behind is zeros
            const uint32_t dst = ring + load_slot * C::STAGE;
#pragma unroll
            for (int i = 0; i < 16 * C::UNITS / 32; ++i) {
                const int x = lane + 32 * i, r = x / C::UNITS, u = x % C::UNITS;
                const size_t from = (row0 + (r < rows ? r : 0)) * D + u * 8;
                const uint32_t to = dst + r * C::PITCH + u * 16, bytes = r < rows ? 16 : 0;
                cp_async16(to, k_pages + from, bytes);
                cp_async16(to + C::TILE, v_pages + from, bytes);
            }
            lk += 16;
        }
        cp_async_commit();
        if (++load_slot == C::STAGES) load_slot = 0;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) issue();

    const int r0 = lane >> 2, c0 = (lane & 3) * 2;         // this thread's rows r0, r0 + 8; columns c0, c0 + 1 of 8
    const uint32_t k_lane = ((lane & 7) + (lane >> 4 & 1) * 8) * C::PITCH + (lane >> 3 & 1) * 16;
    const uint32_t v_lane = (lane & 15) * C::PITCH + (lane >> 4) * 16;
    float* rows_ws = reinterpret_cast<float*>(a.ws);
    float* lse_ws = reinterpret_cast<float*>(a.ws + a.lse_offset);
    int slot = 0;
    FewSegment g;
    while (walk.next(a.plan, a.n_plan, t.h_kv, group, g)) {
        // Q as A operands, and the keys that each row sees
        uint32_t qa[D / 16][4];
        bool live[2];
        int lim[2], tok[2], head[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + 8 * h, rt = r / group;
            live[h] = rt < g.n_tok;
            tok[h] = g.q_tok + (live[h] ? rt : 0);
            head[h] = g.head * group + (live[h] ? r - rt * group : 0);
            lim[h] = g.v.kv;
            if (!(g.v.kind & kKindAll)) {
                const int seen = g.first_pos + rt + 1;
                lim[h] = seen < g.v.kv ? (seen > 0 ? seen : 0) : g.v.kv;
            }
            const uint16_t* from = q + ((size_t)tok[h] * t.h_q + head[h]) * D + c0;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][h] = live[h] ? *reinterpret_cast<const uint32_t*>(from + kk * 16) : 0u;
                qa[kk][2 + h] = live[h] ? *reinterpret_cast<const uint32_t*>(from + kk * 16 + 8) : 0u;
            }
        }
        const int plain = g.v.kind & kKindAll ? g.v.kv : g.first_pos + 1;       // keys that all rows see
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        for (int k = g.k0; k < g.k1; k += 16) {
            cp_async_wait<C::STAGES - 2>();
            __syncwarp();
            const uint32_t ks = ring + slot * C::STAGE + k_lane, vs = ring + slot * C::STAGE + C::TILE + v_lane;
            float x[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                ldmatrix4(ks + kk * 32, b);
                mma_16x8x16(x[0], qa[kk], b[0], b[1]);
                mma_16x8x16(x[1], qa[kk], b[2], b[3]);
            }
            const int last = k + 16 < g.k1 ? k + 16 : g.k1;
            if (k + 16 > plain || last < k + 16) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int left = (lim[h] < last ? lim[h] : last) - k;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (8 * n + c0 + e >= left) x[n][2 * h + e] = -INFINITY;
                }
            }
            float m_new[2];
            bool moves = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mx = fmaxf(fmaxf(x[0][2 * h], x[0][2 * h + 1]), fmaxf(x[1][2 * h], x[1][2 * h + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                m_new[h] = fmaxf(m_run[h], mx * a.scale_log2);
                moves |= live[h] && m_new[h] > m_run[h] + 8.0f;
            }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float f = m_run[h] == -INFINITY ? 0.f : ex2_approx(m_run[h] - m_new[h]);
                    l_run[h] *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][2 * h] *= f;
                        o[i][2 * h + 1] *= f;
                    }
                    m_run[h] = m_new[h];
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float m_ref = m_run[h] == -INFINITY ? 0.f : m_run[h];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2_approx(fmaf(x[n][2 * h], a.scale_log2, -m_ref));
                    const float p1 = ex2_approx(fmaf(x[n][2 * h + 1], a.scale_log2, -m_ref));
                    l_run[h] += p0 + p1;
                    const uint32_t w = pack_bf16x2(p0, p1);
                    hi[2 * n + h] = w;
                    lo[2 * n + h] = pack_bf16x2(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xffff0000u));
                }
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t b[4];
                ldmatrix4_trans(vs + i * 32, b);
                mma_16x8x16(o[2 * i], hi, b[0], b[1]);
                mma_16x8x16(o[2 * i + 1], hi, b[2], b[3]);
                mma_16x8x16(o[2 * i], lo, b[0], b[1]);
                mma_16x8x16(o[2 * i + 1], lo, b[2], b[3]);
            }
            __syncwarp();
            issue();
            if (++slot == C::STAGES) slot = 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = l_run[h];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const float inv = l == 0.f ? 0.f : 1.0f / l;       // NaN stays
            const float lse2 = l == 0.f ? -INFINITY : m_run[h] + log2f(l);
            if (!live[h]) continue;
            const bool joined = g.v.kind & kKindJoined, prefix = g.v.kind & kKindPrefix;
            if (g.whole && !joined) {
                uint32_t* to = reinterpret_cast<uint32_t*>(a.o + ((size_t)tok[h] * t.h_q + head[h]) * D + c0);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) to[i * 4] = pack_bf16x2(o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
                if (c0 == 0) a.lse[(size_t)head[h] * t.n_tokens + tok[h]] = lse2 * 0.693147180559945309f;
                continue;
            }
            const int r = r0 + 8 * h;
            const size_t row = g.whole ? whole_row(t, prefix, tok[h], head[h]) : few_row(t, me, g.from_start ? 1 : 0) + r;
            float* to = rows_ws + row * D + c0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
            if (c0 == 0) {
                lse_ws[row] = lse2;
                if (g.from_start && r % group == 0)
                    a.records[record_at(t, prefix, tok[h], g.head)] =
                        make_record(g.whole, joined, me, g.last, r) | kRecordFew;
            }
        }
    }
    cp_async_wait<0>();
    // the kernel that joins waits for this one, which therefore ends after the one for many rows
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const uint64_t own = a.records[record_at(t, false, tok, kv_head)];
    uint64_t shared = a.records[record_at(t, true, tok, kv_head)];       // meaningless where nothing is shared
    if ((own & kRecordState) == kRecordNone) return;
    if (!(own & kRecordJoined)) shared = kRecordNone;
    auto first = [](uint64_t r) -> int { return (int)(r >> 12 & 0xfffff); };
    auto count = [&](uint64_t r) -> int {
        const uint64_t state = r & kRecordState;
        return state == kRecordNone ? 0 : state == kRecordWhole ? 1 : (int)(r >> 32) - first(r) + 1;
    };
    const int n_own = count(own), parts = n_own + count(shared);
    auto row_of = [&](int p) -> size_t {
        const bool prefix = p >= n_own;
        const uint64_t r = prefix ? shared : own;
        const int i = prefix ? p - n_own : p;
        if ((r & kRecordState) == kRecordWhole) return whole_row(t, prefix, tok, head);
        const int who = first(r) + i, piece = i == 0 ? 1 : 0;
        return (r & kRecordFew ? few_row(t, who, piece) : part_row(who, piece)) + (int)(r >> 4 & 255) + r_head;
    };
    const float* lse = reinterpret_cast<const float*>(a.ws + a.lse_offset);
    const float* rows = reinterpret_cast<const float*>(a.ws) + lane;
    constexpr int E = D / 32, AHEAD = 8;
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
int launch_prefix_t(const PagedMaps& m, PagedArgs a, const PrefixGroups& g, const uint16_t* q, const uint16_t* k_pages,
                    const uint16_t* v_pages, cudaStream_t st)
{
    const PagedTables& t = a.t;
    const PrefixLayout l = prefix_layout(D, t.n_seq, g.n, t.n_tokens, t.h_q, t.h_kv);
    PrefixSeq* plan = reinterpret_cast<PrefixSeq*>(a.ws + l.plan);
    a.plan = plan;
    a.n_plan = g.n + t.n_seq;
    a.records = reinterpret_cast<uint64_t*>(a.ws + l.records);
    a.lse_offset = l.lse;
    a.many_units = reinterpret_cast<const int64_t*>(a.ws + l.many);
    const int n_records = t.n_tokens * t.h_kv;
    const int clearing = n_records / (kPlanThreads * 8);
    prefix_plan_kernel<<<(unsigned)(clearing < 1 ? 1 : clearing < 64 ? clearing : 64), kPlanThreads, 0, st>>>(
        t, a.tpt, a.causal, g, plan, a.records, n_records, reinterpret_cast<int64_t*>(a.ws + l.many));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;

    a.few_waits = 1;
    // batches whose new tokens all together are few rows have no others (the kernel for
    // those has no wait that the test hook could let run out)
    if (!prefix_all_few(a)) {
        constexpr uint32_t smem = PagedCfg<D>::SMEM_PREFIX;
        // (of head groups that the other kernel does not take, single tokens are tiles of few rows)
        const bool fine = a.group > 16 && (int64_t)t.n_tokens * a.group <= (int64_t)kFineRows * t.n_seq;
        auto kern = fine ? paged_attn_kernel<D, true, true> : paged_attn_kernel<D, false, true>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
            return (int)e;
        const int64_t blocks = ((int64_t)t.max_pages * t.page_size + 127) / 128;
        const int64_t row_tiles = ((int64_t)t.n_tokens + a.tpt - 1) / a.tpt;
        const int64_t want = ((2 * row_tiles + a.n_plan) * t.h_kv * blocks + kMinUnits - 1) / kMinUnits;
        int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
        if (want < grid) grid = want;
        if ((e = launch_behind(kern, dim3((unsigned)grid), kThreads, smem, st, m, a)) != cudaSuccess) return (int)e;
        a.few_waits = 0;
    }
    if (a.group <= 16) {
        using C = FewCfg<D>;
        auto kern = prefix_few_kernel<D>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM)) != cudaSuccess)
            return (int)e;
        const int64_t blocks = ((int64_t)t.max_pages * t.page_size + kFewKeys - 1) / kFewKeys;
        const int64_t want = 2 * (int64_t)a.n_plan * t.h_kv * blocks;              // units, at most
        int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
        if (want < grid) grid = want;
        if ((e = launch_behind(kern, dim3((unsigned)grid), C::WARPS * 32, C::SMEM, st, a, q, k_pages, v_pages)) !=
            cudaSuccess)
            return (int)e;
    }
    const int64_t rows = (int64_t)t.n_tokens * t.h_q;
    return (int)launch_behind(prefix_join_kernel<D>, dim3((unsigned)((rows + 3) / 4)), 128, 0, st, a);
}

}  // namespace

size_t prefix_ws_bytes(int d, int n_seq, int n_groups, int64_t n_tokens, int h_q, int h_kv)
{
    return prefix_layout(d, n_seq, n_groups, n_tokens, h_q, h_kv).bytes;
}

bool prefix_all_few(const PagedArgs& a) { return few_rows(a.t.n_tokens, a.group) && !a.inject_timeout; }

int launch_prefix(const PagedMaps& m, const PagedArgs& a, const PrefixGroups& g, const uint16_t* q,
                  const uint16_t* k_pages, const uint16_t* v_pages, cudaStream_t st)
{
    switch (a.d) {
        case 64: return launch_prefix_t<64>(m, a, g, q, k_pages, v_pages, st);
        case 96: return launch_prefix_t<96>(m, a, g, q, k_pages, v_pages, st);
        case 128: return launch_prefix_t<128>(m, a, g, q, k_pages, v_pages, st);
        case 160: return launch_prefix_t<160>(m, a, g, q, k_pages, v_pages, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
