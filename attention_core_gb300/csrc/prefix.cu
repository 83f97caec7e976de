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
// Kernels, launched programmatically one behind the other:
//   plan   turns tables and groups into one list of sequences (prefix_plan.cuh); in small
//          batches the next two make it themselves
//   attend the kernel of paged_attn.cuh over the list's sequences of many rows; rows that
//          have a part of their softmax elsewhere leave as fp32 with their LSE
//   few    the sequences of few rows (a sample's own keys, its single token)
//   join   a warp per row adds its parts up
//
// Measured on one GB300 (64/8 heads of 128 but where said): 64 samples of a prompt of 8192
// keys with up to 500 of their own 48 us (paged_fwd over the same batch: 218), 16 questions
// about 131072 keys 108 us (5.1 TB/s; 820), 6 prompts of up to 4000 keys with 8 samples each, 8/8
// heads of 96, 36 us (86), 2 x 16 sequences with up to 8 drafted tokens over 2000 keys, 16 heads
// of 160, 31 us (85), four samples of 512 keys 12 us in a graph.  What bounds the short ones is
// the chain plan - set-up - first loads (8 us) and the join behind (5 us).
#include <atomic>
#include <chrono>

#include "paged_attn.cuh"

namespace ac {

namespace {

constexpr int kPlanThreads = 1024;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: rows [parts of cut tiles | whole tiles' rows, twice | parts of cut tiles of
// few rows] of d floats, their base-2 LSEs, the records, the plan, its units of many rows
// and the call's stamp.
constexpr int kFewWarps = kPagedMaxCtas * 12;     // of the kernel for few rows, at most
struct PrefixLayout {
    size_t lse, records, plan, many, bytes;
};
__host__ __device__ inline size_t few_row(const PagedTables& t, int warp, int slot)
{
    return (size_t)kPagedMaxCtas * 2 * 128 + 2 * (size_t)t.n_tokens * t.h_q + ((size_t)warp * 2 + slot) * kFewTile;
}
inline PrefixLayout prefix_layout(int d, int n_seq, int n_groups, int64_t n_tokens, int h_q, int h_kv)
{
    const size_t rows = (size_t)kPagedMaxCtas * 2 * 128 + 2 * (size_t)n_tokens * h_q + (size_t)kFewWarps * 2 * kFewTile;
    PrefixLayout l;
    l.lse = align256(rows * d * sizeof(float));
    l.records = align256(l.lse + rows * sizeof(float));
    l.plan = align256(l.records + 2 * (size_t)n_tokens * h_q * sizeof(uint64_t));
    l.many = align256(l.plan + ((size_t)n_seq + n_groups) * sizeof(PrefixSeq));
    l.bytes = l.many + 256;
    return l;
}

// The plan of a batch of more sequences than a block keeps at hand: block 0 plans; all
// blocks clear the records of the sequences' own rows (a token that no tile covers must
// not find an earlier call's).
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PagedTables t, int tpt, int causal,
                                                                   const PrefixGroups gr, PrefixSeq* plan,
                                                                   uint64_t* records, int n_records,
                                                                   int64_t* many_units)
{
    __shared__ int64_t warp_units[kPlanThreads / 32];
    __shared__ unsigned long long many;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0) {
        if (tid == 0) many = 0;
        bool bad = false;
        for (int g = tid; g < gr.n; g += kPlanThreads) bad |= bad_group(gr, g, t.n_seq);
        for (int s = tid; s < t.n_seq; s += kPlanThreads) plan[gr.n + s].page0 = 0;
        bad = __syncthreads_or(bad);
        if (bad && tid == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
        for (int g = warp; g < gr.n; g += kPlanThreads / 32) {
            PrefixSeq shared{};
            if (!bad) {
                const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
                GroupShape shape;
                shape.pages = gr.pages[g] < t.max_pages ? gr.pages[g] : t.max_pages;
                for (int s = s0 + lane; s < s1; s += 32) shape.add(s, read_lengths(t, s, tpt, causal), t.page_shift);
                if (shape.join()) {
                    shared = shape.shared(t.page_shift);
                    for (int s = s0 + lane; s < s1; s += 32) plan[gr.n + s].page0 = shape.pages;
                }
            }
            if (lane == 0) plan[g] = shared;
        }
        __syncthreads();
        const int n = gr.n + t.n_seq;
        int64_t base = 0;
        for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
            const int i = i0 + tid, s = i - gr.n;
            int64_t units = 0;
            PrefixSeq v{};
            if (i < n) {
                v = plan[i];
                if (s >= 0) v = own_part(s, read_lengths(t, s, tpt, causal), v.page0, t.page_shift, causal);
                units = assign(v, t, tpt, &many);
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

// Attention of sequences of few rows (kMostFewRows) over their keys.  A tile of 128 rows
// takes several microseconds from its Q to its O however few of them are used, one after
// another on a processor: 64 samples' own 250 keys took 60 us that way.  Here a warp has a
// piece of a tile of 8 rows by itself, eight on a processor, each with its own ring of
// 16-key steps of K and V (cp.async; 8 KB a step, so that about 100 KB are on their way to
// a processor) and its own softmax.  The scores are formed with the keys as the 16 rows
// and the tile's as the 8 columns of mma.m16n8k16, S^T = K Q^T and O^T += V^T P^T: as many
// products as there are 16 x 16 pieces of K and V, where rows by keys would be twice as
// many, half of them empty.  P goes in as two bf16 terms, as in paged_attn.cuh's tiles of
// few rows.  A step takes a warp about 1400 cycles at d = 96 (the copies' issue 430, scores
// 380, softmax 380, P V 160), so that 152 processors ask for more than HBM gives.
// The units are blocks of 64 keys of (sequence, KV head, row tile), in equal shares for
// all warps; pieces of a tile are joined.  The kernel runs beside the one for many rows:
// that one keeps to as many processors as its part of the work is worth (many_ctas), and
// this one's blocks of lowest number, which are placed first, find the others free.
template <int D>
struct FewCfg {
    static constexpr int UNITS = D / 8;                        // of 16 bytes a row
    static constexpr uint32_t PITCH = (UNITS + 1) * 16;        // odd in 16 bytes: ldmatrix meets no bank twice
    static constexpr uint32_t TILE = 16 * PITCH, STAGE = 2 * TILE;
    static constexpr int COPIES = 16 * UNITS / 32;             // of 16 bytes a lane, for a step's K
    static constexpr int STAGES = D <= 96 ? 4 : D <= 128 ? 3 : 2;
    static constexpr int WARPS = D <= 64 ? 12 : D <= 128 ? 8 : 10;
    static constexpr uint32_t OFF_PLAN = WARPS * STAGES * STAGE, SMEM = OFF_PLAN + sizeof(PlanNear);
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// The plan, in shared memory or in the workspace, where it is read past L1: there a kernel
// wrote it that may still be running (plan_written).
struct PlanView {
    const PrefixSeq* seq;
    int n;
    bool near;
    __device__ __forceinline__ int64_t units(int i) const { return near ? seq[i].few_units : __ldcg(&seq[i].few_units); }
    __device__ __forceinline__ PrefixSeq at(int i) const
    {
        static_assert(sizeof(PrefixSeq) == 32, "two loads");
        if (near) return seq[i];
        union {
            int4 x[2];
            PrefixSeq v;
        } u;
        u.x[0] = __ldcg(reinterpret_cast<const int4*>(seq + i));
        u.x[1] = __ldcg(reinterpret_cast<const int4*>(seq + i) + 1);
        return u.v;
    }
};

// What the kernel for many rows says to this one, which starts beside it: launch_dependents
// orders no memory, so CTA 0 there releases the call's stamp, first as soon as it begins
// and again, one higher, once the plan is written.  Either shows all that came before the
// call, the second the plan; a block that finds the first plans for itself, rather than
// wait (late blocks, which mostly find no share left, read the plan).  Where neither is
// there after several looks, the wait for that kernel's end shows everything.
__device__ __forceinline__ bool plan_written(const PagedArgs& a)
{
    __shared__ uint64_t said;
    if (threadIdx.x == 0) {
        uint64_t seen;
        int looks = 0;
        do
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(a.stamp_at) : "memory");
        while ((seen -= a.stamp) > 1 && ++looks < 64);
        said = seen;
    }
    __syncthreads();
    if (said == 0 && a.n_plan <= kPlanNear) return false;
    if (said != 1) asm volatile("griddepcontrol.wait;" ::: "memory");
    return true;
}

struct FewSegment {
    PrefixSeq v;
    int head, row0, n_rows; // rows of the sequence: new tokens times the head group
    int k0, k1;             // keys [k0, k1)
    bool whole, from_start;
    int last;               // of a cut tile's first piece: the warp of its last one
};

struct FewWalk {
    int64_t at, end, per;
    int s, head, m, b;
    PrefixSeq v;

    // Unit u0 is in the first of the sequences lo .. hi - 1 whose units reach beyond it.
    __device__ __forceinline__ void start(const PlanView& plan, int lo, int hi, int h_kv, int group, int64_t u0, int64_t u1)
    {
        at = u0;
        end = u1;
        const int lane = threadIdx.x & 31;
        while (hi - lo > 32) {                             // 32 candidates a round
            const int step = (hi - lo + 31) / 32;
            const int last = lo + (lane + 1) * step - 1 < hi ? lo + (lane + 1) * step - 1 : hi - 1;
            const uint32_t beyond = __ballot_sync(0xffffffffu, plan.units(last) > u0);
            lo += (__ffs(beyond) - 1) * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        const PrefixSeq c = plan.at(lo + lane < hi ? lo + lane : hi - 1);
        const int src = __ffs(__ballot_sync(0xffffffffu, c.few_units > u0)) - 1;
        s = lo + src;
        v.q0 = __shfl_sync(0xffffffffu, c.q0, src);
        v.nq = __shfl_sync(0xffffffffu, c.nq, src);
        v.kv = __shfl_sync(0xffffffffu, c.kv, src);
        v.row = __shfl_sync(0xffffffffu, c.row, src);
        v.page0 = __shfl_sync(0xffffffffu, c.page0, src);
        v.kind = __shfl_sync(0xffffffffu, c.kind, src);
        v.few_units = __shfl_sync(0xffffffffu, c.few_units, src);
        const int blocks = few_blocks(v.kv), per_head = few_tiles(v.nq * group) * blocks;
        const int64_t rel = u0 - (v.few_units - (int64_t)per_head * h_kv);
        head = (int)quot(rel, per_head);
        const int in_head = (int)(rel - (int64_t)head * per_head);
        m = in_head / blocks;
        b = in_head - m * blocks;
    }

    __device__ __forceinline__ bool next(const PlanView& plan, int h_kv, int group, FewSegment& g)
    {
        if (at >= end) return false;
        int blocks = few_blocks(v.kv);
        if (b >= blocks) {
            b = 0;
            if (++m >= few_tiles(v.nq * group)) {
                m = 0;
                if (++head >= h_kv) {
                    head = 0;
                    do {
                        if (++s >= plan.n) {               // only past the line's end
                            at = end;
                            return false;
                        }
                        v = plan.at(s);
                    } while (!(v.kind & kKindFew));
                    blocks = few_blocks(v.kv);
                }
            }
        }
        const int take = end - at < blocks - b ? (int)(end - at) : blocks - b;
        g.v = v;
        g.head = head;
        g.row0 = m * kFewTile;
        g.n_rows = v.nq * group - g.row0 < kFewTile ? v.nq * group - g.row0 : kFewTile;
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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// The 8 x 8 matrix whose rows the lines of lanes hold, transposed.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
    PlanNear* near = reinterpret_cast<PlanNear*>(smem_raw + C::OFF_PLAN);
    if (a.few_waits) asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool at_hand = a.few_waits ? !a.plan : !plan_written(a);
    if (at_hand) {
        if (a.few_waits) prefetch_table(t);
        plan_near(t, a.tpt, a.causal, a.groups, *near);
    }
    const PlanView plan{at_hand ? near->seq : a.plan, a.n_plan, at_hand};

    // The line's length, and 32 places of it in the same look: this warp's share starts
    // between two of them.
    const int step = (a.n_plan + 31) / 32;
    const int last = (lane + 1) * step < a.n_plan ? (lane + 1) * step - 1 : a.n_plan - 1;
    const int64_t upto = plan.units(last), many = at_hand ? (int64_t)near->many : __ldcg(a.many_units);
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
    load_walk.start(plan, lo, lo + step < a.n_plan ? lo + step : a.n_plan, t.h_kv, group, u0, u1);
    FewWalk walk = load_walk;

    // ---- loads: 16 keys a step, the entries of the page table 32 at a time
    FewSegment lg;
    int lk = 0, window = 0, entry = -1;
    bool loading = load_walk.next(plan, t.h_kv, group, lg);
    auto fetch_entries = [&](int first) {
        window = first;
        const int i = first + lane, n = (lg.v.kv + t.page_size - 1) >> t.page_shift;
        entry = i < n ? t.page_table[(int64_t)lg.v.row * t.max_pages + lg.v.page0 + i] : -1;
    };
    if (loading) {
        lk = lg.k0;
        fetch_entries(lk >> t.page_shift);
    }
    uint32_t copy_to[C::COPIES];                           // where this lane's 16 bytes go in a tile
#pragma unroll
    for (int i = 0; i < C::COPIES; ++i)
        copy_to[i] = (uint32_t)((lane + 32 * i) / C::UNITS) * C::PITCH + (uint32_t)((lane + 32 * i) % C::UNITS) * 16;
    int load_slot = 0;
    auto issue = [&]() {
        while (loading && lk >= lg.k1) {
            loading = load_walk.next(plan, t.h_kv, group, lg);
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
            // (a page's rows of one head are contiguous)
            const uint16_t* kp = k_pages + row0 * D + lane * 8;
            const uint16_t* vp = v_pages + row0 * D + lane * 8;
            if (rows >= 16) {
#pragma unroll
                for (int i = 0; i < C::COPIES; ++i) {
                    cp_async16(dst + copy_to[i], kp + i * 256);
                    cp_async16(dst + copy_to[i] + C::TILE, vp + i * 256);
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::COPIES; ++i) {
                    const bool in = (lane + 32 * i) / C::UNITS < rows;
                    cp_async16(dst + copy_to[i], in ? kp + i * 256 : k_pages, in ? 16 : 0);
                    cp_async16(dst + copy_to[i] + C::TILE, in ? vp + i * 256 : v_pages, in ? 16 : 0);
                }
            }
            lk += 16;
        }
        cp_async_commit();
        if (++load_slot == C::STAGES) load_slot = 0;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) issue();

    // a product's fragments: this thread's line of 8, and its first of two columns of 8
    const int line = lane >> 2, c0 = (lane & 3) * 2;
    const uint32_t k_lane = ((lane & 7) + (lane >> 3 & 1) * 8) * C::PITCH + (lane >> 4) * 16;
    const uint32_t v_lane = ((lane & 7) + (lane >> 4) * 8) * C::PITCH + (lane >> 3 & 1) * 16;
    float* rows_ws = reinterpret_cast<float*>(a.ws);
    float* lse_ws = reinterpret_cast<float*>(a.ws + a.lse_offset);
    int slot = 0;
    FewSegment g;
    while (walk.next(plan, t.h_kv, group, g)) {
        // Q as a B operand
        uint32_t qb[D / 16][2];
        {
            const int r = g.row0 + line, rt = r / group;
            const bool live = line < g.n_rows;
            const uint16_t* from =
                q + ((size_t)(g.v.q0 + (live ? rt : 0)) * t.h_q + g.head * group + (live ? r - rt * group : 0)) * D + c0;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qb[kk][0] = live ? *reinterpret_cast<const uint32_t*>(from + kk * 16) : 0u;
                qb[kk][1] = live ? *reinterpret_cast<const uint32_t*>(from + kk * 16 + 8) : 0u;
            }
        }
        // the two rows whose columns of the scores this thread has, and the keys that they see
        int lim[2];
        bool live[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            live[e] = c0 + e < g.n_rows;
            lim[e] = g.v.kv;
            if (!(g.v.kind & kKindAll)) {
                const int seen = g.v.kv - g.v.nq + (g.row0 + c0 + e) / group + 1;
                lim[e] = seen < g.v.kv ? (seen > 0 ? seen : 0) : g.v.kv;
            }
        }
        // keys that all rows see
        const int plain = g.v.kind & kKindAll ? g.v.kv : g.v.kv - g.v.nq + g.row0 / group + 1;
        float o[D / 16][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        for (int k = g.k0; k < g.k1; k += 16) {
            cp_async_wait<C::STAGES - 2>();
            __syncwarp();
            const uint32_t ks = ring + slot * C::STAGE + k_lane, vs = ring + slot * C::STAGE + C::TILE + v_lane;
            // (several chains of products: one that waits for the one before takes 56 cycles)
            constexpr int CHAINS = 3;
            float x[CHAINS][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t ka[4];
                ldmatrix4(ks + kk * 32, ka);
                mma_16x8x16(x[kk % CHAINS], ka, qb[kk][0], qb[kk][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[0][e] = x[0][e] + x[1][e] + x[2][e];
            const int last = k + 16 < g.k1 ? k + 16 : g.k1;
            const bool masked = k + 16 > plain || last < k + 16;
            uint32_t hi[2], lo[2];
            float m_new[2];
            bool moves = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (masked) {
                    const int left = (lim[e] < last ? lim[e] : last) - k;
                    if (line >= left) x[0][e] = -INFINITY;
                    if (line + 8 >= left) x[0][2 + e] = -INFINITY;
                }
                float mx = fmaxf(x[0][e], x[0][2 + e]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                m_new[e] = fmaxf(m_run[e], mx * a.scale_log2);
                moves |= live[e] && m_new[e] > m_run[e] + 8.0f;
            }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = m_run[e] == -INFINITY ? 0.f : ex2_approx(m_run[e] - m_new[e]);
                    l_run[e] *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[i][e] *= f;
                        o[i][2 + e] *= f;
                    }
                    m_run[e] = m_new[e];
                }
            }
            float p[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m_ref = m_run[e] == -INFINITY ? 0.f : m_run[e];
                p[e] = ex2_approx(fmaf(x[0][e], a.scale_log2, -m_ref));
                p[2 + e] = ex2_approx(fmaf(x[0][2 + e], a.scale_log2, -m_ref));
                l_run[e] += p[e] + p[2 + e];
            }
            // [8 keys x 8 rows] pieces, turned into the B operand of P V's products
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t w = pack_bf16x2(p[2 * n], p[2 * n + 1]);
                hi[n] = movmatrix(w);
                lo[n] = movmatrix(pack_bf16x2(p[2 * n] - __uint_as_float(w << 16),
                                              p[2 * n + 1] - __uint_as_float(w & 0xffff0000u)));
            }
            constexpr int GROUP = D == 64 ? 4 : D / 32;
#pragma unroll
            for (int i0 = 0; i0 < D / 16; i0 += GROUP) {
                uint32_t va[GROUP][4];
#pragma unroll
                for (int i = 0; i < GROUP; ++i) {
                    ldmatrix4_trans(vs + (i0 + i) * 32, va[i]);
                    mma_16x8x16(o[i0 + i], va[i], hi[0], hi[1]);
                }
#pragma unroll
                for (int i = 0; i < GROUP; ++i) mma_16x8x16(o[i0 + i], va[i], lo[0], lo[1]);
            }
            __syncwarp();
            issue();
            if (++slot == C::STAGES) slot = 0;
        }
        const bool joined = g.v.kind & kKindJoined, prefix = g.v.kind & kKindPrefix, done = g.whole && !joined;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_run[e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const float inv = l == 0.f ? 0.f : 1.0f / l;       // NaN stays
            const float lse2 = l == 0.f ? -INFINITY : m_run[e] + log2f(l);
            if (!live[e]) continue;
            const int r = g.row0 + c0 + e, rt = r / group;
            const int tok = g.v.q0 + rt, head = g.head * group + r - rt * group;
            uint64_t* record = a.records + record_at(t, prefix, tok, head);
            if (done) {
                uint16_t* to = a.o + ((size_t)tok * t.h_q + head) * D + line;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t w = pack_bf16x2(o[i][e] * inv, o[i][2 + e] * inv);
                    to[i * 16] = (uint16_t)(w & 0xffffu);
                    to[i * 16 + 8] = (uint16_t)(w >> 16);
                }
                if (line == 0) {
                    a.lse[(size_t)head * t.n_tokens + tok] = lse2 * 0.693147180559945309f;
                    *record = kRecordNone;
                }
                continue;
            }
            const size_t row = g.whole ? whole_row(t, prefix, tok, head) : few_row(t, me, g.from_start ? 1 : 0) + c0 + e;
            float* to = rows_ws + row * D + line;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                to[i * 16] = o[i][e] * inv;
                to[i * 16 + 8] = o[i][2 + e] * inv;
            }
            if (line == 0) {
                lse_ws[row] = lse2;
                if (g.from_start) *record = make_record(g.whole, joined, me, g.last, c0 + e) | kRecordFew;
            }
        }
    }
    cp_async_wait<0>();
    // the kernel that joins waits for this one, which therefore ends after the one for many rows
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A warp per (new token, query head): the parts of the row's own keys' tile, then of
// the group's.  As the join of cut tiles (paged.cu), with the rows found by records.
template <int D, int AHEAD>
__global__ void __launch_bounds__(128) prefix_join_kernel(const PagedArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedTables& t = a.t;
    // a replay of the call from a graph has the same stamp, and may not find it
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.stamp_at = 0;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)t.n_tokens * t.h_q) return;
    const int lane = threadIdx.x & 31;
    const int tok = (int)(row / t.h_q), head = (int)(row % t.h_q);
    const uint64_t own = a.records[record_at(t, false, tok, head)];
    uint64_t shared = a.records[record_at(t, true, tok, head)];       // meaningless where nothing is shared
    if (!a.plan) {
        // no plan's kernel has cleared the records: a token of no sequence finds anything
        bool mine = false;
        for (int s = lane; s < t.n_seq; s += 32) {
            const SeqTable q = read_seq(t, s, a.tpt, a.causal);
            mine |= tok >= q.q0 && tok - q.q0 < q.s.nq;
        }
        if (!__any_sync(0xffffffffu, mine)) return;
    }
    if ((own & kRecordState) == kRecordNone) return;
    if (!(own & kRecordJoined)) shared = kRecordNone;
    // (after a wait that ran out a record may be anything)
    auto sound = [&](uint64_t r) -> bool {
        const uint64_t state = r & kRecordState, who = r >> 12 & 0xfffff, last = r >> 32;
        return state == kRecordNone || state == kRecordWhole ||
               (state == kRecordCut && who <= last && last < (r & kRecordFew ? kFewWarps : kPagedMaxCtas) &&
                (int)(r >> 4 & 255) < (r & kRecordFew ? kFewTile : 128));
    };
    if (!sound(own) || !sound(shared)) return;
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
        return (r & kRecordFew ? few_row(t, who, piece) : part_row(who, piece)) + (int)(r >> 4 & 255);
    };
    const float* lse = reinterpret_cast<const float*>(a.ws + a.lse_offset);
    const float* rows = reinterpret_cast<const float*>(a.ws) + lane;
    constexpr int E = D / 32;
    static_assert(32 % AHEAD == 0, "parts 32 at a time");
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
cudaError_t launch_behind(bool early, void (*kern)(Args...), dim3 grid, int threads, uint32_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Two numbers for each call, from a start that what lies in memory is not (the workspace's
// contents before a call do not matter).
uint64_t next_stamp()
{
    static std::atomic<uint64_t> next{((uint64_t)std::chrono::steady_clock::now().time_since_epoch().count() << 20) | 2};
    return next.fetch_add(2, std::memory_order_relaxed);
}

template <int D>
int launch_prefix_t(const PagedMaps& m, PagedArgs a, const PrefixGroups& g, const uint16_t* q, const uint16_t* k_pages,
                    const uint16_t* v_pages, cudaStream_t st)
{
    const PagedTables& t = a.t;
    const PrefixLayout l = prefix_layout(D, t.n_seq, g.n, t.n_tokens, t.h_q, t.h_kv);
    a.n_plan = g.n + t.n_seq;
    a.groups = g;
    a.records = reinterpret_cast<uint64_t*>(a.ws + l.records);
    a.lse_offset = l.lse;
    a.many_units = reinterpret_cast<int64_t*>(a.ws + l.many);
    a.stamp_at = reinterpret_cast<uint64_t*>(a.many_units) + 1;
    a.stamp = next_stamp();
    a.plan = nullptr;
    a.plan_out = reinterpret_cast<PrefixSeq*>(a.ws + l.plan);
    cudaError_t e;
    if (a.n_plan > kPlanNear) {
        a.plan = a.plan_out;
        const int n_records = t.n_tokens * t.h_q;
        const int clearing = n_records / (kPlanThreads * 8);
        prefix_plan_kernel<<<(unsigned)(clearing < 1 ? 1 : clearing < 64 ? clearing : 64), kPlanThreads, 0, st>>>(
            t, a.tpt, a.causal, g, a.plan_out, a.records, n_records, a.many_units);
        if ((e = cudaGetLastError()) != cudaSuccess) return (int)e;
    }
    bool first = !a.plan;            // the first kernel waits for all that came before
    a.few_waits = 1;
    // batches whose new tokens all together are few rows have no others (the kernel for
    // those has no wait that the test hook could let run out)
    if (!prefix_all_few(a)) {
        constexpr uint32_t smem = PagedCfg<D, true>::SMEM;
        // P of the shared keys in two terms where paged_attn has two for these batches: 64
        // samples 44 -> 48 us, a long document 104 -> 108, drafts 29 -> 31, and O off by
        // 1.7e-3 in the 2-norm, its own rounding, where one term leaves 2.3e-3
        auto kern = fine_batch(a) ? paged_attn_kernel<D, true, true> : paged_attn_kernel<D, false, true>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
            return (int)e;
        const int64_t blocks = ((int64_t)t.max_pages * t.page_size + 127) / 128;
        const int64_t row_tiles = ((int64_t)t.n_tokens + a.tpt - 1) / a.tpt;
        const int64_t want = ((2 * row_tiles + a.n_plan) * t.h_kv * blocks + kMinUnits - 1) / kMinUnits;
        int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
        if (want < grid) grid = want;
        if ((e = launch_behind(!first, kern, dim3((unsigned)grid), kThreads, smem, st, m, a)) != cudaSuccess)
            return (int)e;
        first = false;
        a.few_waits = 0;
    }
    {
        using C = FewCfg<D>;
        auto kern = prefix_few_kernel<D>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM)) != cudaSuccess)
            return (int)e;
        const int64_t blocks = ((int64_t)t.max_pages * t.page_size + kFewKeys - 1) / kFewKeys;
        const int64_t want = (kMostFewRows / kFewTile) * (int64_t)a.n_plan * t.h_kv * blocks;      // units, at most
        int64_t grid = a.num_sms < kPagedMaxCtas ? a.num_sms : kPagedMaxCtas;
        if (want < grid) grid = want;
        PagedArgs few = a;
        if (!few.few_waits) few.plan = a.plan_out;         // the kernel for many rows has written it down
        if ((e = launch_behind(!first, kern, dim3((unsigned)grid), C::WARPS * 32, C::SMEM, st, few, q, k_pages,
                               v_pages)) != cudaSuccess)
            return (int)e;
    }
    // Sixteen parts' loads at a time where few rows have many parts; eight where there are
    // more rows than those blocks' registers let in at once (64 samples: 3 us less).
    const int64_t blocks = ((int64_t)t.n_tokens * t.h_q + 3) / 4;
    auto join = D <= 128 && blocks <= 6 * (int64_t)a.num_sms ? prefix_join_kernel<D, 16> : prefix_join_kernel<D, 8>;
    return (int)launch_behind(true, join, dim3((unsigned)blocks), 128, 0, st, a);
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
