// evict.cu -- eviction from a paged cache by gathered attention weight, on sm_103a.
//
// Per (sequence, KV head) -- a line of n keys -- keep[i] keys stay: the last `recent`,
// the first `first`, and of those between the ones of largest weight, ties to the lower
// index.  They move to the front in their order, with their weights; kept[] says where
// each came from.
//
// select: the H-th largest weight of a line by its bits, 11, 11 and 10 at a time: a
//   histogram of the keys that agree with the bits found so far, summed from the top
//   until H is reached.  The line is read once and kept in shared memory; a line longer
//   than a block's share is split over the blocks of a cluster, whose histograms and
//   counts are added through distributed shared memory.  Then every warp counts what
//   stays of its run of keys by ballots, and places it.  Bound by latency: three
//   histograms, two cluster barriers each.
// move: chunks of 64 kept rows of K and V, 16-byte units through registers.  Bound by
//   the rows' bytes, read and written once.  Rows may move within their own pages: kept
//   row j came from src >= j, so the rows [a, a + 64) that a chunk overwrites are wanted
//   by earlier chunks (and itself) only, those of the kept rows in front of them.  Each
//   chunk is handed out by a counter, earlier ones first, loads without waiting, says so
//   in a flag, and writes once the chunks that read its rows (two at most, by select's
//   ranks) have loaded: a chunk waits only for chunks that were handed out before, which
//   wait for nothing before they have loaded.
#include <cooperative_groups.h>
#include <stddef.h>

#include "kernels.h"
#include "ptx.cuh"

namespace ac {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kMoveRows = 64, kMoveThreads = 256;
constexpr int kBins = 2048;
constexpr int kMostCached = 45056;       // keys that a block keeps in shared memory (176 KB)
constexpr int kSiteEvict = 64;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
__host__ __device__ inline int chunks_of(int64_t n) { return (int)((n + kMoveRows - 1) / kMoveRows); }

// Workspace: [0] the next chunk, [1] the most chunks of a line, [2] a wait has run out; per line the ranks of the
// keys 0, 64, 128, ... (and the line's kept keys at the end); a flag for each chunk.
struct EvictLayout {
    size_t ranks, flags, bytes;
    int per_line;
};
inline EvictLayout evict_layout(int64_t lines, int64_t length)
{
    EvictLayout l;
    l.per_line = chunks_of(length) + 1;
    l.ranks = 256;
    l.flags = align256(l.ranks + (size_t)lines * l.per_line * sizeof(int32_t));
    l.bytes = align256(l.flags + (size_t)lines * l.per_line * sizeof(int32_t));
    return l;
}

// Weights as integers of the same order, NaN below all; the two zeros are one.
__device__ __forceinline__ uint32_t ordered(float w)
{
    const uint32_t u = __float_as_uint(w + 0.0f);
    if (w != w) return 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A line as the tables give it: n keys, of which m stay.
struct Line {
    int n, m, first, recent;
    bool bad;
};
__device__ __forceinline__ Line read_line(const EvictArgs& a, int seq)
{
    const PagedTables& t = a.t;
    Line l;
    const int n = t.kv_lens[seq], keep = a.keep[seq];
    l.bad = n < 0 || n > (int64_t)t.max_pages * t.page_size || keep < 0;
    l.n = l.bad ? 0 : n;
    l.m = keep < l.n ? (l.bad ? 0 : keep) : l.n;
    l.recent = a.recent < l.m ? a.recent : l.m;
    l.first = a.first < l.m - l.recent ? a.first : l.m - l.recent;
    return l;
}

struct SelectShared {
    uint32_t hist[kBins], total[kBins];
    uint32_t warp_sum[kSelectWarps];
    uint32_t bin, above;             // of the pass: where H falls, keys above it
    uint32_t stay[kSelectWarps], tie[kSelectWarps];
    uint32_t block_stay, block_tie;
};

}  // namespace

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a)
{
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ float cache[];
    __shared__ SelectShared sh;
    const PagedTables& t = a.t;
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int line = (int)(blockIdx.x / C), seq = line / t.h_kv;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const size_t length = (size_t)t.max_pages * t.page_size;
    const float* w = a.in + line * length;
    float* out = a.out + line * length;
    int32_t* kept = a.kept + line * length;
    int32_t* ranks = a.ranks + (size_t)line * a.per_line;
    int32_t* flags = a.flags + (size_t)line * a.per_line;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const Line l = read_line(a, seq);
    if (rank == 0 && tid == 0) {
        if (l.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
        ranks[chunks_of(l.n)] = l.m;
        atomicMax(a.most_chunks, chunks_of(l.m));
    }
    for (int c = rank * kSelectThreads + tid; c < chunks_of(l.m); c += C * kSelectThreads) flags[c] = 0;

    // This block's keys [k0, k1), each warp's run a multiple of 64.
    const int run = (int)(((int64_t)l.n + (int64_t)C * kSelectWarps * 64 - 1) / ((int64_t)C * kSelectWarps * 64)) * 64;
    const int64_t share = (int64_t)run * kSelectWarps;
    const int k0 = (int)(rank * share < l.n ? rank * share : l.n), k1 = (int)(k0 + share < l.n ? k0 + share : l.n);
    const bool cached = share <= a.cached;
    if (cached)
        for (int k = k0 + tid; k < k1; k += kSelectThreads) cache[k - k0] = w[k];
    auto at = [&](int k) { return cached ? cache[k - k0] : w[k]; };

    // Candidates [lo, hi), of which `want` stay: the threshold and how many ties of it.
    const int lo = l.first, hi = l.n - l.recent;
    uint32_t want = (uint32_t)(l.m - l.first - l.recent), threshold = 0xffffffffu;
    const bool all = l.m == l.n;
    if (!all && want > 0) {                             // (the same for the whole cluster)
        const int c0 = k0 > lo ? k0 : lo, c1 = k1 < hi ? k1 : hi;
        uint32_t found = 0, mask = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            for (int b = tid; b < kBins; b += kSelectThreads) sh.hist[b] = 0;
            __syncthreads();
            for (int k = c0 + tid; k < c1; k += kSelectThreads) {
                const uint32_t u = ordered(at(k));
                if ((u & mask) == found) atomicAdd(&sh.hist[u >> shift & (bins - 1)], 1u);
            }
            const uint32_t* total = sh.hist;
            if (C > 1) {
                // each block adds up a share of the bins and tells the others
                cluster.sync();
                const int mine = kBins / C;
                for (int b = rank * mine + tid; b < (rank + 1) * mine; b += kSelectThreads) {
                    uint32_t s = 0;
                    for (int r = 0; r < C; ++r) s += cluster.map_shared_rank(sh.hist, r)[b];
                    for (int r = 0; r < C; ++r) cluster.map_shared_rank(sh.total, r)[b] = s;
                }
                cluster.sync();
                total = sh.total;
            } else {
                __syncthreads();
            }
            // sum from the top: thread i has the bins 2047 - 4 i down to 2044 - 4 i
            uint32_t v[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += v[i] = total[kBins - 1 - 4 * tid - i];
            uint32_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            if (lane == 31) sh.warp_sum[warp] = upto;
            __syncthreads();
            for (int i = 0; i < warp; ++i) upto += sh.warp_sum[i];
            uint32_t above = upto - sum;
            if (above < want && want <= upto) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (above < want && want <= above + v[i]) {
                        sh.bin = (uint32_t)(kBins - 1 - 4 * tid - i);
                        sh.above = above;
                    }
                    above += v[i];
                }
            }
            __syncthreads();
            found |= sh.bin << shift;
            mask |= (uint32_t)(bins - 1) << shift;
            want -= sh.above;
            __syncthreads();
        }
        threshold = found;
    } else {
        __syncthreads();
    }
    const uint32_t ties = want;                          // keys at the threshold that stay, the first ones

    // What stays of each warp's run, in order.
    const int w0 = k0 + warp * run < k1 ? k0 + warp * run : k1, w1 = w0 + run < k1 ? w0 + run : k1;
    auto classes = [&](int k, float x, uint32_t& stay, uint32_t& tie) {
        const bool sure = k < w1 && (all || k < lo || k >= hi);
        const bool open = k < w1 && !sure;
        const uint32_t u = open ? ordered(x) : 0u;
        stay = __ballot_sync(0xffffffffu, sure || (open && u > threshold));
        tie = __ballot_sync(0xffffffffu, open && u == threshold);
    };
    uint32_t stays = 0, tied = 0;
    for (int k = w0; k < w1; k += 32) {
        uint32_t s, e;
        classes(k + lane, k + lane < w1 ? at(k + lane) : 0.f, s, e);
        stays += __popc(s);
        tied += __popc(e);
    }
    if (lane == 0) {
        sh.stay[warp] = stays;
        sh.tie[warp] = tied;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t s = 0, e = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            s += sh.stay[i];
            e += sh.tie[i];
        }
        sh.block_stay = s;
        sh.block_tie = e;
    }
    if (C > 1) cluster.sync();                           // also: every block has read its keys
    uint32_t stay0 = 0, tie0 = 0;
    for (int r = 0; r < rank; ++r) {
        stay0 += *cluster.map_shared_rank(&sh.block_stay, r);
        tie0 += *cluster.map_shared_rank(&sh.block_tie, r);
    }
    for (int i = 0; i < warp; ++i) {
        stay0 += sh.stay[i];
        tie0 += sh.tie[i];
    }
    for (int k = w0; k < w1; k += 32) {
        const int key = k + lane;
        const float x = key < w1 ? at(key) : 0.f;
        uint32_t s, e;
        classes(key, x, s, e);
        if (lane == 0 && k % kMoveRows == 0) ranks[k / kMoveRows] = (int32_t)(stay0 + (tie0 < ties ? tie0 : ties));
        const uint32_t before = (1u << lane) - 1;
        const uint32_t tb = tie0 + __popc(e & before);
        const bool stay = (s >> lane & 1) || ((e >> lane & 1) && tb < ties);
        if (stay) {
            const uint32_t j = stay0 + __popc(s & before) + (tb < ties ? tb : ties);
            kept[j] = key;
            if (cached) out[j] = x;
        }
        stay0 += __popc(s);
        tie0 += __popc(e);
    }
    if (C > 1) cluster.sync();                           // no block leaves while another reads its counts
    if (!cached) {
        // a line that no cache holds: the weights move now, rows in front first
        if (C == 1) __syncthreads();
        if (rank) return;
        __threadfence();
        for (int j = 0; j < l.m; j += kSelectThreads) {
            const float x = j + tid < l.m ? w[__ldcg(kept + j + tid)] : 0.f;
            __syncthreads();
            if (j + tid < l.m) out[j + tid] = x;
            __syncthreads();
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a)
{
    constexpr int U = D / 8, LOADS = 2 * kMoveRows * U / kMoveThreads;
    static_assert(2 * kMoveRows * U % kMoveThreads == 0, "units per thread");
    __shared__ int64_t src[kMoveRows], dst[kMoveRows];    // rows of the cache; equal: stays
    __shared__ int ticket, within, wait_first, wait_last, leave;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedTables& t = a.t;
    const int tid = threadIdx.x, lines = t.n_seq * t.h_kv;
    const size_t length = (size_t)t.max_pages * t.page_size;
    const int most = *a.most_chunks;
    for (;;) {
        if (tid == 0) {
            ticket = (int)atomicAdd(a.counter, 1u);
            within = leave = 0;
        }
        __syncthreads();
        const int chunk = ticket / lines, line = ticket - chunk * lines;
        if (chunk >= most) return;
        const int seq = line / t.h_kv, head = line - seq * t.h_kv;
        const Line l = read_line(a, seq);
        if (chunk >= chunks_of(l.m)) {
            __syncthreads();
            continue;
        }
        const int32_t* ranks = a.ranks + (size_t)line * a.per_line;
        int32_t* flags = a.flags + (size_t)line * a.per_line;
        if (tid < kMoveRows) {
            const int j = chunk * kMoveRows + tid;
            int64_t from = 0, to = 0;
            if (j < l.m) {
                const int k = a.kept[line * length + j];
                const int old = t.page_table[(int64_t)seq * t.max_pages + (k >> t.page_shift)];
                const int here = t.page_table[(int64_t)seq * t.max_pages + (j >> t.page_shift)];
                const int page = a.out_table[(int64_t)seq * t.max_pages + (j >> t.page_shift)];
                if (old < 0 || old >= t.n_pages || page < 0 || page >= t.n_pages) {
                    if (t.status) atomicCAS(t.status, 0, kStatusTable);
                } else {
                    from = ((int64_t)old * t.h_kv + head) * t.page_size + (k & (t.page_size - 1));
                    to = ((int64_t)page * t.h_kv + head) * t.page_size + (j & (t.page_size - 1));
                    if (page == here) within = 1;
                }
            }
            src[tid] = from;
            dst[tid] = to;
        } else if (tid == kMoveRows) {
            // the chunks whose rows come from where this one's go
            const int r0 = ranks[chunk], r1 = ranks[chunk + 1 < chunks_of(l.n) ? chunk + 1 : chunks_of(l.n)];
            wait_first = r0 / kMoveRows;
            wait_last = (r1 - 1) / kMoveRows;             // before wait_first: none
            if (r1 <= r0) wait_last = wait_first - 1;
        }
        __syncthreads();
        uint4 x[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = tid + i * kMoveThreads, plane = q / (kMoveRows * U), row = q / U % kMoveRows, u = q % U;
            const uint4* pages = reinterpret_cast<const uint4*>(plane ? a.v_pages : a.k_pages);
            if (src[row] != dst[row]) x[i] = __ldcg(pages + src[row] * U + u);
        }
        __threadfence();                                  // the rows have been read
        __syncthreads();
        if (tid == 0) {
            asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(flags + chunk) : "memory");
            for (int c = within ? wait_first : chunk + 1; c <= wait_last && !leave; ++c) {
                if (c == chunk && !a.inject_timeout) continue;
                const uint64_t began = global_timer_ns();
                for (;;) {
                    int32_t done, over;
                    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(flags + c) : "memory");
                    if (done && !a.inject_timeout) break;
                    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(over) : "l"(a.wait_over) : "memory");
                    if (over || global_timer_ns() - began > a.timeout_ns) {
                        if (!over && t.status) atomicCAS(t.status, 0, 6 | (kSiteEvict << 8));
                        atomicExch(a.wait_over, 1);
                        leave = 1;                        // nothing is written over rows that are still wanted
                        break;
                    }
                }
            }
        }
        __syncthreads();
        if (leave) return;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = tid + i * kMoveThreads, plane = q / (kMoveRows * U), row = q / U % kMoveRows, u = q % U;
            uint4* pages = reinterpret_cast<uint4*>(plane ? a.v_pages : a.k_pages);
            if (src[row] != dst[row]) pages[dst[row] * U + u] = x[i];
        }
        __syncthreads();
    }
}

size_t evict_ws_bytes(int64_t lines, int64_t length) { return evict_layout(lines, length).bytes; }

namespace {

template <int D>
int launch_evict_t(const EvictArgs& args, cudaStream_t st)
{
    EvictArgs a = args;
    const int64_t lines = (int64_t)a.t.n_seq * a.t.h_kv, length = (int64_t)a.t.max_pages * a.t.page_size;
    const EvictLayout lay = evict_layout(lines, length);
    a.counter = reinterpret_cast<uint32_t*>(a.ws);
    a.most_chunks = reinterpret_cast<int32_t*>(a.ws) + 1;
    a.wait_over = reinterpret_cast<int32_t*>(a.ws) + 2;
    a.ranks = reinterpret_cast<int32_t*>(a.ws + lay.ranks);
    a.flags = reinterpret_cast<int32_t*>(a.ws + lay.flags);
    a.per_line = lay.per_line;
    cudaError_t e = cudaMemsetAsync(a.ws, 0, 12, st);
    if (e != cudaSuccess) return (int)e;

    // Blocks per line: more while they have thousands of keys each and the lines leave
    // processors idle.
    int C = 1;
    while (C < 8 && length / C > 4096 && lines * C * 2 <= a.num_sms) C *= 2;
    const int64_t share = ((length + (int64_t)C * kSelectWarps * 64 - 1) / ((int64_t)C * kSelectWarps * 64)) * 64 * kSelectWarps;
    a.cached = (int)(share < kMostCached ? share : kMostCached);
    const uint32_t smem = (uint32_t)a.cached * sizeof(float);
    if ((e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
        return (int)e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(lines * C));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a)) != cudaSuccess) return (int)e;

    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    const int64_t chunks = lines * chunks_of(length), most = (int64_t)a.num_sms * 6;
    cfg.gridDim = dim3((unsigned)(chunks < most ? chunks : most));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    return (int)cudaLaunchKernelEx(&cfg, evict_move_kernel<D>, a);
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t st)
{
    switch (a.d) {
        case 64: return launch_evict_t<64>(a, st);
        case 96: return launch_evict_t<96>(a, st);
        case 128: return launch_evict_t<128>(a, st);
        case 160: return launch_evict_t<160>(a, st);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace ac
