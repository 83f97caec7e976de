// prefix_plan.cuh -- the plan of a batch whose sequences share their first pages: one list
// of sequences (PrefixSeq, paged_sched.cuh), each group's shared keys first, then each
// sequence's own.
#pragma once
#include "kernels.h"
#include "paged_sched.cuh"

namespace ac {

namespace {

// Sequences of few rows (new tokens times the head group): the kernel for those has them,
// in tiles of 8 rows and blocks of 64 keys.  More rows than 32 would read K and V more
// than four times (from L2); 128 rows of the other kernel read them once.
constexpr int kFewTile = 8, kMostFewRows = 32, kFewKeys = 64;
__host__ __device__ inline bool few_rows(int nq, int group) { return nq > 0 && nq <= kMostFewRows && nq * group <= kMostFewRows; }
__host__ __device__ inline int few_tiles(int rows) { return (rows + kFewTile - 1) / kFewTile; }
__host__ __device__ inline int few_blocks(int kv) { return kv > 0 ? (int)(((uint32_t)kv + kFewKeys - 1) / kFewKeys) : 1; }

// What a group shares in fact: whole pages that all its sequences with new tokens hold
// before their first, so that no row's mask ends inside them; a group of one shares
// nothing.  A whole warp asks, its lanes for some of the sequences each.
struct GroupShape {
    int members = 0, pages, q0 = INT32_MAX, q1 = 0, row = INT32_MAX;
    // len: first token, new tokens, keys
    __device__ __forceinline__ void add(int s, const int4& len, int page_shift)
    {
        if (len.y <= 0) return;
        const int old = len.z > len.y ? (len.z - len.y) >> page_shift : 0;
        pages = old < pages ? old : pages;
        ++members;
        q0 = len.x < q0 ? len.x : q0;
        q1 = len.x + len.y > q1 ? len.x + len.y : q1;
        row = s < row ? s : row;
    }
    __device__ __forceinline__ bool join()
    {
        members = __reduce_add_sync(0xffffffffu, members);
        pages = __reduce_min_sync(0xffffffffu, pages);
        q0 = __reduce_min_sync(0xffffffffu, q0);
        q1 = __reduce_max_sync(0xffffffffu, q1);
        row = __reduce_min_sync(0xffffffffu, row);
        return members > 1 && pages > 0;
    }
    __device__ __forceinline__ PrefixSeq shared(int page_shift) const
    {
        return PrefixSeq{q0, q1 - q0, pages << page_shift, row, 0, kKindAll | kKindPrefix | kKindJoined, 0};
    }
};
__device__ __forceinline__ PrefixSeq own_part(int s, const int4& len, int pages, int page_shift, int causal)
{
    if (len.y <= 0) pages = 0;
    return PrefixSeq{len.x, len.y, len.z - (pages << page_shift), s, pages,
                     (causal ? 0 : kKindAll) | (pages ? kKindJoined : 0), 0};
}
__device__ __forceinline__ int4 read_lengths(const PagedTables& t, int s, int tpt, int causal)
{
    const SeqTable q = read_seq(t, s, tpt, causal);
    if (q.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
    return make_int4(q.q0, q.s.nq, q.s.kv, 0);
}
__device__ __forceinline__ bool bad_group(const PrefixGroups& gr, int g, int n_seq)
{
    const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
    return s0 < 0 || s1 < s0 || s1 > n_seq || gr.pages[g] < 0;
}

// Who has sequence v, and its units there.
__device__ __forceinline__ int64_t assign(PrefixSeq& v, const PagedTables& t, int tpt, unsigned long long* many)
{
    const int group = t.h_q / t.h_kv;
    if (few_rows(v.nq, group)) {
        v.kind |= kKindFew;
        return (int64_t)few_tiles(v.nq * group) * few_blocks(v.kv) * t.h_kv;
    }
    if (v.nq > 0) {
        const SeqShape q{v.nq, v.kv, tpt, !(v.kind & kKindAll)};
        atomicAdd(many, (unsigned long long)q.units(q.tiles()) * t.h_kv);
    }
    return 0;
}

// The page table towards L2, a line a thread, while the plan is made: whoever loads keys
// waits for its entries next.
__device__ __forceinline__ void prefetch_table(const PagedTables& t)
{
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (at * 32 < (int64_t)t.n_seq * t.max_pages)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(t.page_table + at * 32) : "memory");
}

// The plan of a batch of few sequences, which each block makes for itself in shared
// memory: 2 us, where a kernel for it and the wait for that one cost 5.
constexpr int kPlanNear = 128;                       // sequences and groups together
struct PlanNear {
    PrefixSeq seq[kPlanNear];
    int4 len[kPlanNear];                             // .w: shared pages
    int64_t warp_units[kPlanNear / 32];
    unsigned long long many;                         // units of the kernel for many rows
};
// All threads of the block, kPlanNear at least.
__device__ __forceinline__ void plan_near(const PagedTables& t, int tpt, int causal, const PrefixGroups& gr, PlanNear& p)
{
    const int tid = threadIdx.x, lane = tid & 31, n = gr.n + t.n_seq;
    if (tid < t.n_seq) p.len[tid] = read_lengths(t, tid, tpt, causal);
    const bool bad_one = tid < gr.n && bad_group(gr, tid, t.n_seq);
    if (tid == 0) p.many = 0;
    const bool bad = __syncthreads_or(bad_one);
    if (bad && tid == 0 && t.status) atomicCAS(t.status, 0, kStatusTable);
    for (int g = tid >> 5; g < gr.n; g += (int)blockDim.x / 32) {
        PrefixSeq shared{};
        if (!bad) {
            const int s0 = gr.starts[g], s1 = gr.starts[g + 1];
            GroupShape shape;
            shape.pages = gr.pages[g] < t.max_pages ? gr.pages[g] : t.max_pages;
            for (int s = s0 + lane; s < s1; s += 32) shape.add(s, p.len[s], t.page_shift);
            if (shape.join()) {
                shared = shape.shared(t.page_shift);
                for (int s = s0 + lane; s < s1; s += 32) p.len[s].w = shape.pages;
            }
        }
        if (lane == 0) p.seq[g] = shared;
    }
    __syncthreads();
    PrefixSeq v{};
    int64_t units = 0;
    if (tid < n) {
        const int s = tid - gr.n;
        v = s < 0 ? p.seq[tid] : own_part(s, p.len[s], p.len[s].w, t.page_shift, causal);
        units = assign(v, t, tpt, &p.many);
    }
    int64_t upto = units;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31 && tid < kPlanNear) p.warp_units[tid / 32] = upto;
    __syncthreads();
    if (tid < n) {
        for (int w = 0; w < tid / 32; ++w) upto += p.warp_units[w];
        v.few_units = upto;
        p.seq[tid] = v;
    }
    __syncthreads();
}

}  // namespace

}  // namespace ac
