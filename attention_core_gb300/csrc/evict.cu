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
//   stays of its run of keys, four a lane at a time, and places it.  Bound by the passes'
//   latency: three histograms (two copies of the first, whose bins weights crowd into) and
//   two passes over the keys; 30 us for 512 lines of up to 8192 keys and for 8 of 131072.
//   Two blocks a processor: with four, the waiting blocks of the next kernel found their
//   places unevenly, and that kernel took 25 us longer.
// move: chunks of 64 kept rows of K and V, 16-byte units through registers.  Bound by
//   the rows' bytes, read and written once.  Rows may move within their own pages: kept
//   row j came from src >= j, so the rows [a, a + 64) that a chunk overwrites are wanted
//   by earlier chunks (and itself) only, those of the kept rows in front of them.  Each
//   chunk is handed out by a counter, earlier ones first, loads without waiting, says so
//   in a flag, and writes once the chunks that read its rows (two at most, by select's
//   ranks) have loaded: a chunk waits only for chunks that were handed out before, which
//   wait for nothing before they have loaded.
// Measured on one GB300, 8 KV heads of 128: 64 sequences of up to 8192 keys cut to 2048
// 196 us (the move 165 of them, 6.4 TB/s), one of 131072 keys cut to 32768 74 us, one of
// 600 keys 7 us in a graph.
#include <cooperative_groups.h>
#include <stddef.h>

#include "kernels.h"
#include "ptx.cuh"

namespace ac {

namespace cg = cooperative_groups;

namespace {

constexpr int kMoveRows = 64, kMoveThreads = 256;
constexpr int kBins = 2048;
constexpr int kMostCached = 45056;       // keys that a block keeps in shared memory (176 KB)
constexpr int kSiteEvict = 64;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
__host__ __device__ inline int chunks_of(int64_t n) { return (int)((n + kMoveRows - 1) / kMoveRows); }

// Workspace: [0] the next chunk, [1] a wait has run out; per line the ranks of the
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

struct alignas(16) SelectShared {
    uint32_t hist[2][kBins];         // two copies in the first pass
    uint32_t warp_sum[32];
    uint32_t bin, above;             // of the pass: where H falls, keys above it
    uint32_t warp_tie[32];
    uint32_t block_stay, block_tie;
};

}  // namespace

// T threads: 512, two blocks a processor; 1024 where lines are split over clusters, whose
// processors have one block each.
template <int T>
__global__ void __launch_bounds__(T, 1024 / T) evict_select_kernel(const EvictArgs a)
{
    constexpr int kSelectThreads = T, kSelectWarps = T / 32, B = kBins / T;     // B bins a thread
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) float cache[];        // keys; behind them, in clusters, the added histogram
    __shared__ SelectShared sh;
    const PagedTables& t = a.t;
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int line = (int)(blockIdx.x / C), seq = line / t.h_kv;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const size_t length = (size_t)t.max_pages * t.page_size;
    const float* w = a.in + line * length;
    int32_t* ranks = a.ranks + (size_t)line * a.per_line;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const Line l = read_line(a, seq);
    if (rank == 0 && tid == 0) {
        if (l.bad && t.status) atomicCAS(t.status, 0, kStatusTable);
        ranks[chunks_of(l.n)] = l.m;
        if (line == 0) {
            *a.counter = 0u;
            *a.wait_over = 0;
        }
    }
    {
        int32_t* flags = a.flags + (size_t)line * a.per_line;
        for (int c = rank * kSelectThreads + tid; c < chunks_of(l.m); c += C * kSelectThreads) flags[c] = 0;
    }

    // This block's keys [k0, k1), each warp's run a multiple of 128: four keys a thread at a
    // time.  (What lies between the line's n and its row's end is read, and not used.)
    const int run = (int)(((int64_t)l.n + (int64_t)C * kSelectWarps * 128 - 1) / ((int64_t)C * kSelectWarps * 128)) * 128;
    const int64_t share = (int64_t)run * kSelectWarps;
    const int k0 = (int)(rank * share < l.n ? rank * share : l.n), k1 = (int)(k0 + share < l.n ? k0 + share : l.n);
    const bool cached = share <= a.cached;
    for (int b = tid; b < 2 * kBins; b += kSelectThreads) sh.hist[0][b] = 0;
    if (cached)
        for (int k = k0 + 4 * tid; k < k1; k += 4 * kSelectThreads)
            *reinterpret_cast<float4*>(cache + (k - k0)) = *reinterpret_cast<const float4*>(w + k);
    auto at = [&](int k) -> float4 {
        return *reinterpret_cast<const float4*>(cached ? cache + (k - k0) : w + k);
    };
    __syncthreads();

    // Candidates [lo, hi), of which `want` stay: the threshold and how many ties of it.
    const int lo = l.first, hi = l.n - l.recent;
    uint32_t want = (uint32_t)(l.m - l.first - l.recent), threshold = 0xffffffffu;
    const bool all = l.m == l.n;
    if (!all && want > 0) {                             // (the same for the whole cluster)
        uint32_t found = 0;
        const int c0 = lo < k0 ? k0 : lo & ~3, c1 = k1 < hi ? k1 : hi;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            if (pass > 0) {
                for (int b = tid; b < kBins; b += kSelectThreads) sh.hist[0][b] = 0;
                __syncthreads();
            }
            {
                // two copies of the first pass's: weights crowd in few of its bins
                uint32_t* hist = sh.hist[pass == 0 ? warp & 1 : 0];
                for (int k = c0 + 4 * tid; k < c1; k += 4 * kSelectThreads) {
                    const float4 x = at(k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = ordered(e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w);
                        const bool open = k + e >= lo && k + e < c1;
                        if (open && (pass == 0 || u >> (shift + (pass == 1 ? 11 : 10)) == found >> (shift + (pass == 1 ? 11 : 10))))
                            atomicAdd(hist + (u >> shift & (bins - 1)), 1u);
                    }
                }
            }
            __syncthreads();
            const uint32_t* total = sh.hist[0];
            const bool second = pass == 0;              // copy to be added
            if (C > 1) {
                // each block adds up a share of the bins and tells the others
                uint32_t* sum_of = reinterpret_cast<uint32_t*>(cache) + a.cached;
                cluster.sync();
                const int mine = kBins / C;
                for (int b = rank * mine + tid; b < (rank + 1) * mine; b += kSelectThreads) {
                    uint32_t s = 0;
                    for (int r = 0; r < C; ++r) {
                        const uint32_t* h = cluster.map_shared_rank(&sh.hist[0][0], r);
                        s += h[b] + (second ? h[kBins + b] : 0u);
                    }
                    for (int r = 0; r < C; ++r) cluster.map_shared_rank(sum_of, r)[b] = s;
                }
                cluster.sync();
                total = sum_of;
            }
            // sum from the top: thread i has the B bins down from 2047 - B i
            uint32_t v[B], sum = 0;
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int b = kBins - 1 - B * tid - i;
                v[i] = total[b];
                if (C == 1 && second) v[i] += sh.hist[1][b];
                sum += v[i];
            }
            uint32_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            if (lane == 31) sh.warp_sum[warp] = upto;
            __syncthreads();
            uint32_t before = lane < warp ? sh.warp_sum[lane] : 0u;
            before = __reduce_add_sync(0xffffffffu, before);
            upto += before;
            uint32_t above = upto - sum;
            if (above < want && want <= upto) {
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    if (above < want && want <= above + v[i]) {
                        sh.bin = (uint32_t)(kBins - 1 - B * tid - i);
                        sh.above = above;
                    }
                    above += v[i];
                }
            }
            __syncthreads();
            found |= sh.bin << shift;
            want -= sh.above;
            __syncthreads();
        }
        threshold = found;
    }
    const uint32_t ties = want;                          // keys at the threshold that stay, the first ones

    // What stays of each warp's run, in order: keys that stay for certain, and ties.
    const int w0 = k0 + warp * run < k1 ? k0 + warp * run : k1, w1 = w0 + run < k1 ? w0 + run : k1;
    // bits e and e + 4: key k + e stays, is a tie
    auto classes = [&](int k, const float4& x) -> uint32_t {
        uint32_t c = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = k + e < w1, sure = all || k + e < lo || k + e >= hi;
            const uint32_t u = ordered(e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w);
            if (in && (sure || u > threshold)) c |= 1u << e;
            if (in && !sure && u == threshold) c |= 16u << e;
        }
        return c;
    };
    uint32_t stays = 0, tied = 0;
    for (int k = w0 + 4 * lane; k < w1; k += 128) {
        const uint32_t c = classes(k, at(k));
        stays += __popc(c & 15u);
        tied += __popc(c >> 4);
    }
    stays = __reduce_add_sync(0xffffffffu, stays);
    tied = __reduce_add_sync(0xffffffffu, tied);
    if (lane == 0) {
        sh.warp_sum[warp] = stays;
        sh.warp_tie[warp] = tied;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t s = __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? sh.warp_sum[lane] : 0u);
        const uint32_t e = __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? sh.warp_tie[lane] : 0u);
        if (lane == 0) {
            sh.block_stay = s;
            sh.block_tie = e;
        }
    }
    uint32_t stay0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u);
    uint32_t tie0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_tie[lane] : 0u);
    if (C > 1) cluster.sync();                           // also: every block has read its keys
    for (int r = 0; r < rank; ++r) {
        stay0 += *cluster.map_shared_rank(&sh.block_stay, r);
        tie0 += *cluster.map_shared_rank(&sh.block_tie, r);
    }
    float* out = a.out + line * length;
    int32_t* kept = a.kept + line * length;
    for (int k = w0 + 4 * lane; k - 4 * lane < w1; k += 128) {
        const float4 x = k < w1 ? at(k) : make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t c = classes(k, x);
        uint32_t upto = __popc(c & 15u) | __popc(c >> 4) << 16;          // of 128 keys: no carry
        const uint32_t own = upto;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t step = __shfl_sync(0xffffffffu, upto, 31);
        uint32_t s = stay0 + ((upto - own) & 0xffffu), e = tie0 + ((upto - own) >> 16);
        if ((lane & 15) == 0 && k < w1) ranks[k / kMoveRows] = (int32_t)(s + (e < ties ? e : ties));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool tie = c >> (4 + i) & 1;
            if ((c >> i & 1) || (tie && e < ties)) {
                const uint32_t j = s + (e < ties ? e : ties);
                kept[j] = k + i;
                if (cached) out[j] = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
            }
            s += c >> i & 1;
            e += tie;
        }
        stay0 += step & 0xffffu;
        tie0 += step >> 16;
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
    __shared__ int ticket, within, wait_first, wait_last, leave, most;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedTables& t = a.t;
    const int tid = threadIdx.x, lines = t.n_seq * t.h_kv;
    const size_t length = (size_t)t.max_pages * t.page_size;
    // chunks of the longest line
    if (tid == 0) most = 0;
    __syncthreads();
    int longest = 0;
    for (int s = tid; s < t.n_seq; s += kMoveThreads) {
        const int m = read_line(a, s).m;
        longest = m > longest ? m : longest;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((tid & 31) == 0) atomicMax(&most, chunks_of(longest));
    __syncthreads();
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
    a.wait_over = reinterpret_cast<int32_t*>(a.ws) + 1;
    a.ranks = reinterpret_cast<int32_t*>(a.ws + lay.ranks);
    a.flags = reinterpret_cast<int32_t*>(a.ws + lay.flags);
    a.per_line = lay.per_line;
    cudaError_t e;
    // Blocks per line: more while they have thousands of keys each and the lines leave
    // processors idle.
    int C = 1;
    while (C < 8 && length / C > 4096 && lines * C * 2 <= a.num_sms) C *= 2;
    const int threads = C > 1 ? 1024 : 512;
    const int64_t step = (int64_t)threads * 4;             // keys that a block has at a time
    const int64_t share = (length + C * step - 1) / (C * step) * step;
    a.cached = (int)(share < kMostCached ? share : kMostCached);
    const uint32_t smem = (uint32_t)a.cached * sizeof(float) + (C > 1 ? kBins * sizeof(uint32_t) : 0);
    auto select = C > 1 ? evict_select_kernel<1024> : evict_select_kernel<512>;
    // The limit is the kernel's, not the call's: a size that follows the lengths would be
    // lowered by another thread's shorter lines between here and this call's launch.
    constexpr int most_smem = kMostCached * sizeof(float) + kBins * sizeof(uint32_t);
    if ((e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem)) != cudaSuccess)
        return (int)e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(lines * C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, select, a)) != cudaSuccess) return (int)e;

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
