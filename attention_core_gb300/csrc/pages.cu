// pages.cu -- page copies inside a paged key/value cache on sm_103a.
//
// Page dst <- page src of every plane, for a list of (src, dst) pairs that
// travels as a kernel parameter, so the host's list needs no device copy and no
// lifetime.  Bound by HBM: each copied byte is read and written once.  A block
// copies a 16 KB piece of one page of one plane, every thread four 16-byte
// units with all its loads in flight before the first store.  Measured: 400 pages
// of 128 KB in each of 16 planes 246 us (6.8 TB/s, the rate of a plain copy); one
// page of 32 KB in 16 planes 2.3 us in a graph.
#include "kernels.h"

namespace ac {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;   // 16-byte units per thread

template <int N>
struct PairList {
    int2 p[N];
};

}  // namespace

template <int N>
__global__ void __launch_bounds__(kCopyThreads)
page_copy_kernel(uint4* pages, int64_t plane_units, int64_t page_units, int pieces,
                 const __grid_constant__ PairList<N> list)
{
    const int2 pr = list.p[blockIdx.x / pieces];
    uint4* plane = pages + blockIdx.y * plane_units;
    const uint4* src = plane + pr.x * page_units;
    uint4* dst = plane + pr.y * page_units;
    const int64_t u0 = (int64_t)(blockIdx.x % pieces) * (kCopyThreads * kCopyUnits) + threadIdx.x;
    uint4 v[kCopyUnits];
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
        if (u0 + i * kCopyThreads < page_units) v[i] = __ldcs(src + u0 + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
        if (u0 + i * kCopyThreads < page_units) __stcs(dst + u0 + i * kCopyThreads, v[i]);
}

namespace {

template <int N>
int launch_list(uint4* pages, int64_t n_planes, int64_t plane_units, int64_t page_units, const int32_t* pairs, int n,
                cudaStream_t st)
{
    PairList<N> list;
    for (int i = 0; i < n; ++i) list.p[i] = make_int2(pairs[2 * i], pairs[2 * i + 1]);
    for (int i = n; i < N; ++i) list.p[i] = make_int2(0, 0);
    const int pieces = (int)((page_units + kCopyThreads * kCopyUnits - 1) / (kCopyThreads * kCopyUnits));
    const dim3 grid((unsigned)(n * pieces), (unsigned)n_planes);
    page_copy_kernel<N><<<grid, kCopyThreads, 0, st>>>(pages, plane_units, page_units, pieces, list);
    return (int)cudaGetLastError();
}

}  // namespace

// A list of up to 32 pairs is a 256-byte parameter; longer ones go out 960 at a
// time (7.7 KB).
int launch_page_copy(void* pages, int64_t n_planes, int64_t plane_bytes, int64_t page_bytes, const int32_t* pairs,
                     int64_t n_pairs, cudaStream_t st)
{
    uint4* base = static_cast<uint4*>(pages);
    for (int64_t i = 0; i < n_pairs;) {
        const int64_t left = n_pairs - i;
        const int n = (int)(left < 960 ? left : 960);
        const auto launch = n <= 32 ? launch_list<32> : launch_list<960>;
        const int e = launch(base, n_planes, plane_bytes / 16, page_bytes / 16, pairs + 2 * i, n, st);
        if (e) return e;
        i += n;
    }
    return 0;
}

}  // namespace ac
