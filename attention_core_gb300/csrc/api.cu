// api.cu -- the C ABI declared in include/attn_core.h: argument checks,
// TMA tensor-map encoding and kernel launches.  No device memory is
// allocated here; the caller owns every buffer.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/attn_core.h"
#include "kernels.h"
#include "philox.cuh"
#include "tile.cuh"

namespace {

using ac::kBlockRows;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int get_encoder()
{
    if (g_encode) return ATTN_CORE_OK;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr) return ATTN_CORE_ERR_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return ATTN_CORE_OK;
}

// 0: not checked yet, 1: sm_103, -1: other.
int g_dev_ok[128];

int check_device()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_CORE_ERR_CUDA;
    if (dev < 0 || dev >= 128) return ATTN_CORE_ERR_UNSUPPORTED;
    if (g_dev_ok[dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return ATTN_CORE_ERR_CUDA;
        g_dev_ok[dev] = (major == 10 && minor == 3) ? 1 : -1;
    }
    return g_dev_ok[dev] == 1 ? ATTN_CORE_OK : ATTN_CORE_ERR_UNSUPPORTED;
}

int g_dev_sms[128];

int device_sms(int* out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return ATTN_CORE_ERR_CUDA;
    if (g_dev_sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return ATTN_CORE_ERR_CUDA;
        g_dev_sms[dev] = n;
    }
    *out = g_dev_sms[dev];
    return ATTN_CORE_OK;
}

bool supported_d(int d) { return d == 64 || d == 96 || d == 128 || d == 160; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Keys per KV head: s_kv, or s when s_kv is 0.
int keys_of(const attn_core_params* p) { return p->s_kv ? p->s_kv : p->s; }

int check_params(const attn_core_params* p)
{
    if (p == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->b <= 0 || p->h_q <= 0 || p->h_kv <= 0 || p->s <= 0 || p->d <= 0 || p->s_kv < 0)
        return ATTN_CORE_ERR_INVALID_ARG;
    if (p->h_q % p->h_kv != 0) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->causal != 0 && p->causal != 1) return ATTN_CORE_ERR_INVALID_ARG;
    if (!(p->p_drop >= 0.0f && p->p_drop < 1.0f)) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->offset >> 32) return ATTN_CORE_ERR_INVALID_ARG;
    if (isnan(p->scale) || isinf(p->scale)) return ATTN_CORE_ERR_INVALID_ARG;
    // Counter words and grid sizes are 32-bit.
    const int64_t n_bh = (int64_t)p->b * p->h_q;
    const int64_t n_blk = ((int64_t)p->s + kBlockRows - 1) / kBlockRows;
    const int64_t n_blk_k = ((int64_t)keys_of(p) + kBlockRows - 1) / kBlockRows;
    if (n_bh * n_blk >= (int64_t)INT32_MAX || n_bh * n_blk_k >= (int64_t)INT32_MAX ||
        (int64_t)p->s * n_bh >= ((int64_t)1 << 40))
        return ATTN_CORE_ERR_INVALID_ARG;
    return ATTN_CORE_OK;
}

// Dropout threshold of the attention core on an 8-bit draw: round(p * 256), at
// most 255; an element is dropped iff its draw is below it.
uint32_t drop_threshold(float p)
{
    if (!(p > 0.0f)) return 0u;
    long long t = llround((double)p * 256.0);
    if (t > 255) t = 255;
    if (t < 0) t = 0;
    return (uint32_t)t;
}

// The dropout + layer norm block's threshold on a 16-bit draw: round(p * 65536),
// at most 65535.
uint32_t drop_threshold16(float p)
{
    if (!(p > 0.0f)) return 0u;
    long long t = llround((double)p * 65536.0);
    if (t > 65535) t = 65535;
    if (t < 0) t = 0;
    return (uint32_t)t;
}

ac::CommonArgs common_args(const attn_core_params* p)
{
    ac::CommonArgs c{};
    c.s = p->s;
    c.s_k = keys_of(p);
    c.h_q = p->h_q;
    c.h_kv = p->h_kv;
    c.n_blk = (p->s + kBlockRows - 1) / kBlockRows;
    c.n_blk_k = (c.s_k + kBlockRows - 1) / kBlockRows;
    c.n_bh = p->b * p->h_q;
    c.causal = p->causal;
    const float scale = (p->scale > 0.0f) ? p->scale : 1.0f / sqrtf((float)p->d);
    c.scale = scale;
    c.scale_log2 = scale * 1.44269504088896340736f;
    c.thr = drop_threshold(p->p_drop);
    c.keep_scale = 1.0f / (1.0f - (float)c.thr / 256.0f);
    c.seed_lo = (uint32_t)(p->seed & 0xffffffffu);
    c.seed_hi = (uint32_t)(p->seed >> 32);
    ac::philox_round_keys(c.seed_lo, c.seed_hi, c.rk);
    c.offset = (uint32_t)p->offset;
    c.status = p->dev_status;
    c.timeout_ns = (uint64_t)(p->wait_timeout_ms ? p->wait_timeout_ms : 2000u) * 1000000ull;
    c.inject_timeout = (p->flags & ATTN_CORE_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    c.bh0 = 0;
    c.lse_stride = p->s;
    return c;
}

// 3-D map over `heads` x `s` rows of d bf16 values, row r of head h at
// ptr + h * head_stride + r * row_stride elements: box = one column chunk of
// `rows` rows of one head, swizzled to match the shared-memory tile layout.
// [heads, s, d] tensors have row_stride d and head_stride s * d; one sequence
// of a packed [tokens, heads, d] batch has row_stride heads * d and
// head_stride d.
int encode_map_strided(CUtensorMap* m, const void* ptr, int d, int s, int64_t heads, int64_t row_stride,
                       int64_t head_stride, int rows)
{
    const int cw = (d % 64 == 0) ? 64 : 32;
    const CUtensorMapSwizzle sw = (cw == 64) ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)s, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2, (cuuint64_t)head_stride * 2};
    cuuint32_t box[3] = {(cuuint32_t)cw, (cuuint32_t)rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_CORE_OK : ATTN_CORE_ERR_CUDA;
}

int encode_map(CUtensorMap* m, const void* ptr, int cw, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box)
{
    const CUtensorMapSwizzle sw = (cw == 64) ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides,
                          box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_CORE_OK : ATTN_CORE_ERR_CUDA;
}

// 4-D map over packed rows [tokens][kv heads][group][d] bf16: box = cw columns of the
// `group` rows of one KV head of `tpt` tokens.
int encode_map_tokens(CUtensorMap* m, const void* ptr, int cw, int d, int group, int kv_heads, int64_t tokens, int tpt)
{
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)group, (cuuint64_t)kv_heads, (cuuint64_t)tokens};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)group * d * 2, (cuuint64_t)kv_heads * group * d * 2};
    const cuuint32_t box[4] = {(cuuint32_t)cw, (cuuint32_t)group, 1, (cuuint32_t)tpt};
    return encode_map(m, ptr, cw, 4, dims, strides, box);
}

// 3-D map over pages [page and KV head][page_size][d] bf16: box = cw columns of up to
// 128 rows of one page.
int encode_map_pages(CUtensorMap* m, const void* ptr, int cw, int d, int page_size, int64_t pages)
{
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)pages};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)page_size * d * 2};
    const cuuint32_t box[3] = {(cuuint32_t)cw, (cuuint32_t)(page_size < kBlockRows ? page_size : kBlockRows), 1};
    return encode_map(m, ptr, cw, 3, dims, strides, box);
}

// Where the query-side (Q, O, dO, dQ) and key-side (K, V, dK, dV) rows of one
// launch live, and where its LSE rows go.
struct Geometry {
    int64_t q_heads, kv_heads;              // map heads: b * h_q and b * h_kv, or h_q and h_kv
    int64_t q_row, q_head, kv_row, kv_head; // strides in elements
    int64_t lse_stride;                     // LSE elements from one query head to the next
    uint32_t bh0;                           // Philox head-index offset
    int64_t q_rows, k_rows;                 // rows per map head: s and s_kv, or a packed
                                            // batch's total query and key counts
    int64_t ws_stride;                      // backward workspace rows per query head
    const int32_t* cu_q;                    // a packed batch's device sequence tables,
    const int32_t* cu_k;                    // or null
};

Geometry padded_geometry(const attn_core_params* p, int sk)
{
    Geometry g;
    g.q_heads = (int64_t)p->b * p->h_q;
    g.kv_heads = (int64_t)p->b * p->h_kv;
    g.q_row = g.kv_row = p->d;
    g.q_head = (int64_t)p->s * p->d;
    g.kv_head = (int64_t)sk * p->d;
    g.lse_stride = p->s;
    g.bh0 = 0;
    g.q_rows = p->s;
    g.k_rows = sk;
    g.ws_stride = ((int64_t)p->s + kBlockRows - 1) / kBlockRows * kBlockRows;
    g.cu_q = g.cu_k = nullptr;
    return g;
}

size_t padded_rows(const attn_core_params* p)
{
    const size_t n_blk = ((size_t)p->s + kBlockRows - 1) / kBlockRows;
    return (size_t)p->b * p->h_q * n_blk * kBlockRows;
}

// Bytes of the keep bits the dQ kernel hands to the dK/dV kernel (p > 0,
// d <= 128).  For d = 160 the dK/dV kernel is bound by its products, not by
// its row threads, so drawing the mask there again costs no time, while
// writing the bits would cost the dQ kernel some: that case draws twice.
size_t mask_bytes(const attn_core_params* p)
{
    if (drop_threshold(p->p_drop) == 0 || p->d > 128 || (p->flags & ATTN_CORE_FLAG_REDRAW_MASK)) return 0;
    // the hand-over layout covers the square causal pattern; causal
    // cross-attention draws the mask twice
    if (p->causal && keys_of(p) != p->s) return 0;
    const ac::CommonArgs c = common_args(p);
    return sizeof(uint32_t) * ac::mask_ws_words(c);
}

int record(void** ev, int idx, cudaStream_t st)
{
    if (!ev) return ATTN_CORE_OK;
    return cudaEventRecord(reinterpret_cast<cudaEvent_t>(ev[idx]), st) == cudaSuccess ? ATTN_CORE_OK
                                                                                       : ATTN_CORE_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* attn_core_strerror(int code)
{
    switch (code & 0xff) {
        case ATTN_CORE_OK: return "ok";
        case ATTN_CORE_ERR_INVALID_ARG: return "invalid argument";
        case ATTN_CORE_ERR_UNSUPPORTED: return "unsupported head dimension or device";
        case ATTN_CORE_ERR_MISALIGNED: return "pointer not aligned (16 bytes; workspace 256 bytes)";
        case ATTN_CORE_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
        case ATTN_CORE_ERR_CUDA: return "CUDA error";
        case ATTN_CORE_ERR_DEVICE_TIMEOUT: return "a kernel wait ran past its time limit";
        case ATTN_CORE_ERR_DEVICE_TABLE: return "a device table held an entry out of range";
        default: return "unknown error";
    }
}

int attn_core_stored_bytes(const attn_core_params* p, attn_core_bytes* out)
{
    int rc = check_params(p);
    if (rc) return rc;
    if (!out) return ATTN_CORE_ERR_INVALID_ARG;
    const int64_t s = p->s, sk = keys_of(p), b = p->b, a = p->h_q, akv = p->h_kv, d = p->d;
    const int64_t h = a * d;
    out->layer_selective = 34 * s * b * h;
    out->layer_none = out->layer_selective + 5 * a * s * s * b;
    out->layer_full = 2 * s * b * h;
    out->core_scores_avoided = 5 * a * s * sk * b;
    out->core_kept = 2 * d * b * (2 * a * s + 2 * akv * sk);
    out->core_recompute_state = 4 * b * a * s + 16;
    return ATTN_CORE_OK;
}

size_t attn_core_bwd_workspace_bytes(const attn_core_params* p)
{
    if (check_params(p)) return 0;
    return 2 * sizeof(float) * padded_rows(p) + mask_bytes(p);
}

}  // extern "C"

namespace {

// One forward launch over the geometry g (pointers at the launch's first row).
int fwd_launch(const attn_core_params* p, const Geometry& g, const void* q, const void* k, const void* v, void* o,
               float* lse, cudaStream_t st)
{
    int rc;
    const int sk = keys_of(p);
    (void)sk;
    CUtensorMap tq, tk, tv, to;
    if ((rc = encode_map_strided(&tq, q, p->d, (int)g.q_rows, g.q_heads, g.q_row, g.q_head, 128)) ||
        (rc = encode_map_strided(&tk, k, p->d, (int)g.k_rows, g.kv_heads, g.kv_row, g.kv_head, 128)) ||
        (rc = encode_map_strided(&tv, v, p->d, (int)g.k_rows, g.kv_heads, g.kv_row, g.kv_head, 128)) ||
        (rc = encode_map_strided(&to, o, p->d, (int)g.q_rows, g.q_heads, g.q_row, g.q_head, 128)))
        return rc;
    ac::FwdArgs a{};
    a.c = common_args(p);
    a.c.bh0 = g.bh0;
    a.c.lse_stride = g.lse_stride;
    a.c.cu_q = g.cu_q;
    a.c.cu_k = g.cu_k;
    a.c.ws_stride = g.ws_stride;
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    a.o_head_stride = g.q_head;
    a.o_row_stride = g.q_row;
    if ((rc = device_sms(&a.num_sms))) return rc;
    if ((rc = record(p->timing_events, 0, st))) return rc;
    if (ac::launch_fwd(p->d, a.c.thr != 0, tq, tk, tv, to, a, st) != 0) return ATTN_CORE_ERR_CUDA;
    return record(p->timing_events, 1, st);
}

}  // namespace

extern "C" {

int attn_core_fwd(const attn_core_params* p, const void* q, const void* k, const void* v, void* o, float* lse,
                  void* stream)
{
    int rc = check_params(p);
    if (rc) return rc;
    if (!q || !k || !v || !o || !lse) return ATTN_CORE_ERR_INVALID_ARG;
    if (!supported_d(p->d)) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return ATTN_CORE_ERR_MISALIGNED;
    if ((rc = check_device())) return rc;
    if ((rc = get_encoder())) return rc;
    return fwd_launch(p, padded_geometry(p, keys_of(p)), q, k, v, o, lse, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace {

// Workspace bytes of one backward launch: the two row statistics and (when
// shared) the keep bits, rounded up to 256 bytes.
size_t launch_ws_bytes(const attn_core_params* p, bool share_mask)
{
    const size_t b = 2 * sizeof(float) * padded_rows(p) + (share_mask ? mask_bytes(p) : 0);
    return (b + 255) & ~(size_t)255;
}

// One backward launch (dQ, then dK/dV) over the geometry g; `workspace` holds
// launch_ws_bytes(p, share_mask) bytes.  share_mask: the workspace also holds
// the keep bits, which the dQ kernel writes and the dK/dV kernel reads;
// otherwise the dK/dV kernel draws the mask again from Philox.
int bwd_launch(const attn_core_params* p, const Geometry& g, const void* q, const void* k, const void* v,
               const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
               bool share_mask, cudaStream_t st)
{
    int rc;
    const int bq = ac::dkdv_query_tile(p->d);
    const int bn = ac::dq_key_tile(p->d);
    const int sk = keys_of(p);
    auto qmap = [&](CUtensorMap* m, const void* ptr, int rows) {
        return encode_map_strided(m, ptr, p->d, (int)g.q_rows, g.q_heads, g.q_row, g.q_head, rows);
    };
    auto kmap = [&](CUtensorMap* m, const void* ptr, int rows) {
        return encode_map_strided(m, ptr, p->d, (int)g.k_rows, g.kv_heads, g.kv_row, g.kv_head, rows);
    };
    CUtensorMap tq128, tdo128, to128, tdq128, tqb, tdob, tk, tv, tkb, tvb, tdk, tdv;
    if ((rc = qmap(&tq128, q, 128)) || (rc = qmap(&tdo128, dout, 128)) || (rc = qmap(&to128, o, 128)) ||
        (rc = qmap(&tdq128, dq, 128)) ||
        (rc = qmap(&tqb, q, bq)) || (rc = qmap(&tdob, dout, bq)) || (rc = kmap(&tk, k, 128)) ||
        (rc = kmap(&tv, v, 128)) || (rc = kmap(&tkb, k, bn)) || (rc = kmap(&tvb, v, bn)) ||
        (rc = kmap(&tdk, dk, 128)) || (rc = kmap(&tdv, dv, 128)))
        return rc;
    ac::BwdArgs a{};
    a.c = common_args(p);
    a.c.bh0 = g.bh0;
    a.c.lse_stride = g.lse_stride;
    a.c.cu_q = g.cu_q;
    a.c.cu_k = g.cu_k;
    a.c.ws_stride = g.ws_stride;
    a.s_pad = a.c.n_blk * kBlockRows;
    const size_t ws_rows = (size_t)g.q_heads * (size_t)g.ws_stride;
    a.o = static_cast<const uint16_t*>(o);
    a.dout = static_cast<const uint16_t*>(dout);
    a.lse = lse;
    a.lse2_ws = static_cast<float*>(workspace);
    a.delta_ws = static_cast<float*>(workspace) + ws_rows;
    a.mask_ws = (share_mask && g.cu_q == nullptr && mask_bytes(p) != 0)
                    ? reinterpret_cast<uint32_t*>(static_cast<float*>(workspace) + 2 * ws_rows)
                    : nullptr;
    a.dq = static_cast<uint16_t*>(dq);
    a.dk = static_cast<uint16_t*>(dk);
    a.dv = static_cast<uint16_t*>(dv);
    a.q_head_stride = g.q_head;
    a.q_row_stride = g.q_row;
    a.kv_head_stride = g.kv_head;
    a.kv_row_stride = g.kv_row;
    a.d = p->d;
    if ((rc = device_sms(&a.num_sms))) return rc;
    const bool drop = a.c.thr != 0;
    if ((rc = record(p->timing_events, 0, st))) return rc;
    if (ac::launch_bwd_dq(p->d, drop, tq128, tkb, tvb, tdo128, to128, tdq128, a, st) != 0) return ATTN_CORE_ERR_CUDA;
    if ((rc = record(p->timing_events, 1, st)) || (rc = record(p->timing_events, 2, st))) return rc;
    if (ac::launch_bwd_dkdv(p->d, drop, tqb, tk, tv, tdob, tdk, tdv, a, st) != 0) return ATTN_CORE_ERR_CUDA;
    // Causal with more keys than queries: keys from the end of the last query
    // block on are seen by no query (top-left alignment) and the dK/dV kernel
    // skips their blocks, so their gradients are set to zero here.
    const int64_t kz = (int64_t)a.c.n_blk * kBlockRows;
    if (g.cu_q == nullptr && p->causal && sk > kz) {
        const size_t row_bytes = (size_t)g.kv_row * sizeof(uint16_t);
        for (void* t : {dk, dv}) {
            uint8_t* base = static_cast<uint8_t*>(t) + (size_t)kz * row_bytes;
            cudaError_t e;
            if (g.kv_head == p->d) {        // token-major rows: all heads of a row are adjacent
                e = cudaMemsetAsync(base, 0, (size_t)(sk - kz) * row_bytes, st);
            } else {                        // head-major: rows kz .. sk - 1 of every head
                e = cudaMemset2DAsync(base, (size_t)g.kv_head * sizeof(uint16_t), 0, (size_t)(sk - kz) * row_bytes,
                                      (size_t)g.kv_heads, st);
            }
            if (e != cudaSuccess) return ATTN_CORE_ERR_CUDA;
        }
    }
    return record(p->timing_events, 3, st);
}

// The backward of the padded layout.
int bwd_impl(const attn_core_params* p, const void* q, const void* k, const void* v, const void* o,
             const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
             size_t workspace_bytes, bool share_mask, void* stream)
{
    int rc = check_params(p);
    if (rc) return rc;
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return ATTN_CORE_ERR_INVALID_ARG;
    if (!supported_d(p->d)) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return ATTN_CORE_ERR_MISALIGNED;
    const size_t need = 2 * sizeof(float) * padded_rows(p) + (share_mask ? mask_bytes(p) : 0);
    if (workspace_bytes < need) return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device())) return rc;
    if ((rc = get_encoder())) return rc;
    return bwd_launch(p, padded_geometry(p, keys_of(p)), q, k, v, o, lse, dout, dq, dk, dv, workspace, share_mask,
                      reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int attn_core_bwd_recompute(const attn_core_params* p, const void* q, const void* k, const void* v, const void* o,
                            const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    return bwd_impl(p, q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, true, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Variable-length (packed) batches: one launch per kernel over the whole batch.
// The kernels take the n_seq sequences as a batch of n_seq elements of the
// longest sequence's length and read each tile's own lengths and first rows
// from the device copies of the sequence tables.
namespace {

struct VarlenShape {
    int64_t total_q, total_k;
    int32_t max_q, max_k;
    const int32_t* cu_q_dev;
    const int32_t* cu_k_dev;
};

// Checks the host sequence tables and the device copies' presence.
int check_varlen(const attn_core_varlen_params* vp, VarlenShape* out)
{
    if (vp == nullptr || vp->n_seq <= 0 || vp->cu_seqlens_q == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if (vp->cu_seqlens_q_dev == nullptr || (vp->cu_seqlens_k != nullptr && vp->cu_seqlens_k_dev == nullptr))
        return ATTN_CORE_ERR_INVALID_ARG;
    if (vp->base.timing_events != nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if ((int64_t)vp->n_seq * vp->base.h_q >= (int64_t)INT32_MAX) return ATTN_CORE_ERR_INVALID_ARG;
    const int32_t* cq = vp->cu_seqlens_q;
    const int32_t* ck = vp->cu_seqlens_k ? vp->cu_seqlens_k : cq;
    if (cq[0] != 0 || ck[0] != 0) return ATTN_CORE_ERR_INVALID_ARG;
    int32_t max_q = 0, max_k = 0;
    for (int i = 0; i < vp->n_seq; ++i) {
        const int32_t lq = cq[i + 1] - cq[i], lk = ck[i + 1] - ck[i];
        if (lq < 0 || lk < 0 || (lq > 0 && lk == 0)) return ATTN_CORE_ERR_INVALID_ARG;
        if (lq > max_q) max_q = lq;
        if (lk > max_k) max_k = lk;
    }
    out->total_q = cq[vp->n_seq];
    out->total_k = ck[vp->n_seq];
    if (out->total_q >= (int64_t)INT32_MAX - 132 * (int64_t)vp->n_seq - 4 || out->total_k >= (int64_t)INT32_MAX)
        return ATTN_CORE_ERR_INVALID_ARG;
    out->max_q = max_q;
    out->max_k = max_k;
    out->cu_q_dev = vp->cu_seqlens_q_dev;
    out->cu_k_dev = vp->cu_seqlens_k ? vp->cu_seqlens_k_dev : vp->cu_seqlens_q_dev;
    return ATTN_CORE_OK;
}

// The batch as one launch: n_seq elements of the longest sequence's length.
attn_core_params batch_params(const attn_core_varlen_params* vp, const VarlenShape& vs)
{
    attn_core_params ps = vp->base;
    ps.b = vp->n_seq;
    ps.s = vs.max_q;
    ps.s_kv = vs.max_k;
    return ps;
}

// Packed [tokens, heads, d] tensors: one map head per attention head, rows of
// the whole batch.
Geometry packed_geometry(const attn_core_varlen_params* vp, const VarlenShape& vs)
{
    Geometry g;
    g.q_heads = vp->base.h_q;
    g.kv_heads = vp->base.h_kv;
    g.q_row = (int64_t)vp->base.h_q * vp->base.d;
    g.kv_row = (int64_t)vp->base.h_kv * vp->base.d;
    g.q_head = g.kv_head = vp->base.d;
    g.lse_stride = vs.total_q;
    g.bh0 = 0;
    g.q_rows = vs.total_q;
    g.k_rows = vs.total_k;
    g.ws_stride = ((vs.total_q + 3) & ~(int64_t)3) + 132 * (int64_t)vp->n_seq;   // see packed_ws_row0
    g.cu_q = vs.cu_q_dev;
    g.cu_k = vs.cu_k_dev;
    return g;
}

size_t varlen_ws_bytes(const attn_core_varlen_params* vp, const VarlenShape& vs)
{
    const size_t rows = (size_t)((vs.total_q + 3) & ~(int64_t)3) + 132 * (size_t)vp->n_seq;
    const size_t b = 2 * sizeof(float) * (size_t)vp->base.h_q * rows;
    return (b + 255) & ~(size_t)255;
}

}  // namespace

extern "C" {

size_t attn_core_bwd_varlen_workspace_bytes(const attn_core_varlen_params* vp)
{
    VarlenShape vs;
    if (check_varlen(vp, &vs)) return 0;
    return varlen_ws_bytes(vp, vs);
}

int attn_core_fwd_varlen(const attn_core_varlen_params* vp, const void* q, const void* k, const void* v, void* o,
                         float* lse, void* stream)
{
    VarlenShape vs;
    int rc = check_varlen(vp, &vs);
    if (rc) return rc;
    if (!q || !k || !v || !o || !lse) return ATTN_CORE_ERR_INVALID_ARG;
    if (!supported_d(vp->base.d)) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return ATTN_CORE_ERR_MISALIGNED;
    if (vs.max_q == 0) return ATTN_CORE_OK;          // no queries: nothing to compute
    const attn_core_params ps = batch_params(vp, vs);
    if ((rc = check_params(&ps))) return rc;
    if ((rc = check_device())) return rc;
    if ((rc = get_encoder())) return rc;
    return fwd_launch(&ps, packed_geometry(vp, vs), q, k, v, o, lse, reinterpret_cast<cudaStream_t>(stream));
}

int attn_core_bwd_varlen(const attn_core_varlen_params* vp, const void* q, const void* k, const void* v,
                         const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                         void* workspace, size_t workspace_bytes, void* stream)
{
    VarlenShape vs;
    int rc = check_varlen(vp, &vs);
    if (rc) return rc;
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return ATTN_CORE_ERR_INVALID_ARG;
    if (!supported_d(vp->base.d)) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return ATTN_CORE_ERR_MISALIGNED;
    if (workspace_bytes < varlen_ws_bytes(vp, vs)) return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (vs.max_q == 0) {
        // no query sees any key: every key's gradients are zero
        const size_t nb = (size_t)vs.total_k * vp->base.h_kv * vp->base.d * sizeof(uint16_t);
        if (nb && (cudaMemsetAsync(dk, 0, nb, st) != cudaSuccess || cudaMemsetAsync(dv, 0, nb, st) != cudaSuccess))
            return ATTN_CORE_ERR_CUDA;
        return ATTN_CORE_OK;
    }
    const attn_core_params ps = batch_params(vp, vs);
    if ((rc = check_params(&ps))) return rc;
    if ((rc = check_device())) return rc;
    if ((rc = get_encoder())) return rc;
    return bwd_launch(&ps, packed_geometry(vp, vs), q, k, v, o, lse, dout, dq, dk, dv, workspace, false, st);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Dropout + residual add + layer norm.
namespace {

int check_dal(const attn_core_dal_params* p)
{
    if (p == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->n_rows <= 0 || p->hidden <= 0 || p->hidden % 8 != 0) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->hidden > ac::kDalMaxHidden) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!(p->p_drop >= 0.0f && p->p_drop < 1.0f)) return ATTN_CORE_ERR_INVALID_ARG;
    if (!(p->eps > 0.0f) || isinf(p->eps)) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->offset >> 32) return ATTN_CORE_ERR_INVALID_ARG;
    return ATTN_CORE_OK;
}

ac::DalArgs dal_args(const attn_core_dal_params* p)
{
    ac::DalArgs a{};
    a.n_rows = p->n_rows;
    a.hidden = p->hidden;
    a.eps = p->eps;
    a.thr = drop_threshold16(p->p_drop);
    a.keep_scale = 1.0f / (1.0f - (float)a.thr / 65536.0f);
    a.seed_lo = (uint32_t)(p->seed & 0xffffffffu);
    a.seed_hi = (uint32_t)(p->seed >> 32);
    ac::philox_round_keys(a.seed_lo, a.seed_hi, a.rk);
    a.offset = (uint32_t)p->offset;
    a.status = p->dev_status;
    a.timeout_ns = (uint64_t)(p->wait_timeout_ms ? p->wait_timeout_ms : 2000u) * 1000000ull;
    return a;
}

int dal_partial_rows(const attn_core_dal_params* p)
{
    return p->n_rows < ac::kDalMaxPartial ? p->n_rows : ac::kDalMaxPartial;
}

}  // namespace

extern "C" {

int attn_core_dropout_add_ln_fwd(const attn_core_dal_params* p, const void* x, const void* residual,
                                 const float* gamma, const float* beta, void* z, void* y, float* mean,
                                 float* rstd, void* stream)
{
    int rc = check_dal(p);
    if (rc) return rc;
    if (!x || !residual || !gamma || !beta || !z || !y || !mean || !rstd) return ATTN_CORE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(beta) || !aligned16(z) ||
        !aligned16(y))
        return ATTN_CORE_ERR_MISALIGNED;
    if ((rc = check_device())) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    ac::DalArgs a = dal_args(p);
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.gamma = gamma;
    a.beta = beta;
    a.z = static_cast<uint16_t*>(z);
    a.y = static_cast<uint16_t*>(y);
    a.mean = mean;
    a.rstd = rstd;
    return ac::launch_dal_fwd(a, sms, reinterpret_cast<cudaStream_t>(stream)) ? ATTN_CORE_ERR_CUDA : ATTN_CORE_OK;
}

size_t attn_core_dropout_add_ln_bwd_workspace_bytes(const attn_core_dal_params* p)
{
    if (check_dal(p)) return 0;
    return 2 * sizeof(float) * (size_t)p->hidden * (size_t)dal_partial_rows(p);
}

int attn_core_dropout_add_ln_bwd(const attn_core_dal_params* p, const void* dy, const void* dz_next,
                                 const void* z, const float* mean, const float* rstd, const float* gamma,
                                 void* dx, void* d_residual, float* dgamma, float* dbeta, void* workspace,
                                 size_t workspace_bytes, void* stream)
{
    int rc = check_dal(p);
    if (rc) return rc;
    if (!dy || !z || !mean || !rstd || !gamma || !dx || !d_residual || !dgamma || !dbeta || !workspace)
        return ATTN_CORE_ERR_INVALID_ARG;
    if (!aligned16(dy) || (dz_next && !aligned16(dz_next)) || !aligned16(z) || !aligned16(gamma) ||
        !aligned16(dx) || !aligned16(d_residual) || !aligned16(workspace))
        return ATTN_CORE_ERR_MISALIGNED;
    if (workspace_bytes < attn_core_dropout_add_ln_bwd_workspace_bytes(p)) return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL;
    if ((rc = check_device())) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    ac::DalArgs a = dal_args(p);
    a.gamma = gamma;
    a.z = static_cast<uint16_t*>(const_cast<void*>(z));
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = static_cast<const uint16_t*>(dy);
    a.dz_next = static_cast<const uint16_t*>(dz_next);
    a.dx = static_cast<uint16_t*>(dx);
    a.d_residual = static_cast<uint16_t*>(d_residual);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.partial = static_cast<float*>(workspace);
    return ac::launch_dal_bwd(a, sms, reinterpret_cast<cudaStream_t>(stream)) ? ATTN_CORE_ERR_CUDA : ATTN_CORE_OK;
}

}  // extern "C"

// GeLU of the layer's MLP.
extern "C" {

int attn_core_gelu_fwd(int64_t n, const void* x, void* y, void* stream)
{
    if (n <= 0 || n % 8 != 0 || !x || !y) return ATTN_CORE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y)) return ATTN_CORE_ERR_MISALIGNED;
    int rc = check_device();
    if (rc) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    return ac::launch_gelu_fwd(static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), n, sms,
                               reinterpret_cast<cudaStream_t>(stream))
               ? ATTN_CORE_ERR_CUDA
               : ATTN_CORE_OK;
}

int attn_core_gelu_bwd(int64_t n, const void* x, const void* dy, void* dx, void* stream)
{
    if (n <= 0 || n % 8 != 0 || !x || !dy || !dx) return ATTN_CORE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx)) return ATTN_CORE_ERR_MISALIGNED;
    int rc = check_device();
    if (rc) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    return ac::launch_gelu_bwd(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dy),
                               static_cast<uint16_t*>(dx), n, sms, reinterpret_cast<cudaStream_t>(stream))
               ? ATTN_CORE_ERR_CUDA
               : ATTN_CORE_OK;
}

}  // extern "C"

// Backward for callers that cannot allocate device memory.  Its workspace is a
// fixed array of this library's own, 2 * kNoAllocMaxRows fp32 values (8 MiB),
// which every GPU that loads the library holds until the process exits.  In
// host code the array's name is only a host-side stand-in: every call looks up
// its device address for the current device with cudaGetSymbolAddress (which
// allocates nothing) and passes that address to the kernels, so the address is
// never stale, not even after the device's context has been reset.
static constexpr size_t kNoAllocMaxRows = (size_t)1 << 20;
static __device__ __align__(256) float g_noalloc_scratch[2 * kNoAllocMaxRows];

extern "C" {

int attn_core_bwd_recompute_noalloc(const attn_core_params* p, const void* q, const void* k, const void* v,
                                    const void* o, const float* lse, const void* dout, void* dq, void* dk,
                                    void* dv, void* stream)
{
    int rc = check_params(p);
    if (rc) return rc;
    if (padded_rows(p) > kNoAllocMaxRows) return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL;
    void* addr = nullptr;
    if (cudaGetSymbolAddress(&addr, g_noalloc_scratch) != cudaSuccess || addr == nullptr) return ATTN_CORE_ERR_CUDA;
    // The fixed array holds the two row statistics only; the dK/dV kernel draws
    // its own mask.
    return bwd_impl(p, q, k, v, o, lse, dout, dq, dk, dv, addr, sizeof(float) * 2 * kNoAllocMaxRows, false,
                    stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Rotary positions.
static_assert(sizeof(ac::RopeTable) == sizeof(attn_core_rope_table), "the table is passed as it is");
static_assert(ac::kStatusTable == ATTN_CORE_ERR_DEVICE_TABLE, "status code");

namespace {

constexpr double kTwoPi = 6.283185307179586;
constexpr int kMaxHeads = 65535;    // heads may be shared out over as many rows of blocks

bool positive(double x) { return x > 0.0 && !isinf(x); }

int check_rope_table(const attn_core_rope_table* t)
{
    if (t == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if (t->d < 8 || t->d > 512 || t->d % 8 || t->rot_dim < 8 || t->rot_dim > 256 || t->rot_dim > t->d ||
        t->rot_dim % 8 || (t->interleaved != 0 && t->interleaved != 1))
        return ATTN_CORE_ERR_INVALID_ARG;
    return ATTN_CORE_OK;
}

// Strides of one tensor: rows 16-byte aligned and, of an output, apart: the
// dimensions in the order of their strides each step over the whole of the
// smaller ones.
int check_rope_strides(const int64_t (&st)[3], int64_t b, int64_t h, int64_t s, int64_t d, bool output)
{
    const int64_t n[3] = {b, h, s};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0) return ATTN_CORE_ERR_INVALID_ARG;
        if (st[i] % 8) return ATTN_CORE_ERR_MISALIGNED;
        if (st[i] > ((int64_t)1 << 42)) return ATTN_CORE_ERR_INVALID_ARG;
    }
    if (!output) return ATTN_CORE_OK;
    int64_t span = d;
    bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
    for (int k = 0; k < 3; ++k) {
        int least = -1;
        for (int i = 0; i < 3; ++i)
            if (!used[i] && (least < 0 || st[i] < st[least])) least = i;
        if (least < 0) break;
        used[least] = true;
        if (st[least] < span) return ATTN_CORE_ERR_INVALID_ARG;
        span += st[least] * (n[least] - 1);
    }
    return ATTN_CORE_OK;
}

int rope_call(const attn_core_rope_params* p, const attn_core_rope_table* t, const void* q, const void* k, void* yq,
              void* yk, float sign, void* stream)
{
    int rc = check_rope_table(t);
    if (rc) return rc;
    if (p == nullptr || p->b <= 0 || p->s < 0 || p->h_q < 0 || p->h_kv < 0 || p->h_q + (int64_t)p->h_kv == 0 ||
        (int64_t)p->b * p->s >= (int64_t)INT32_MAX - kBlockRows)     // tokens, counted in whole blocks
        return ATTN_CORE_ERR_INVALID_ARG;
    if (p->h_q + (int64_t)p->h_kv > kMaxHeads) return ATTN_CORE_ERR_UNSUPPORTED;
    if ((p->h_q && (!q || !yq)) || (p->h_kv && (!k || !yk))) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->h_q && ((rc = check_rope_strides(p->q_stride, p->b, p->h_q, p->s, t->d, q == yq)) ||
                   (rc = check_rope_strides(p->yq_stride, p->b, p->h_q, p->s, t->d, true))))
        return rc;
    if (p->h_kv && ((rc = check_rope_strides(p->k_stride, p->b, p->h_kv, p->s, t->d, k == yk)) ||
                    (rc = check_rope_strides(p->yk_stride, p->b, p->h_kv, p->s, t->d, true))))
        return rc;
    // an output may be its own input, but neither the other input nor the other output
    if (p->h_q && p->h_kv && p->s > 0 && (yq == yk || yq == k || yk == q)) return ATTN_CORE_ERR_INVALID_ARG;
    // in place means the same element at the same place
    for (int i = 0; i < 3; ++i)
        if ((p->h_q && q == yq && p->q_stride[i] != p->yq_stride[i]) ||
            (p->h_kv && k == yk && p->k_stride[i] != p->yk_stride[i]))
            return ATTN_CORE_ERR_INVALID_ARG;
    if ((p->h_q && (!aligned16(q) || !aligned16(yq))) || (p->h_kv && (!aligned16(k) || !aligned16(yk))) ||
        (reinterpret_cast<uintptr_t>(p->positions) & 3u))
        return ATTN_CORE_ERR_MISALIGNED;
    if (p->s == 0) return ATTN_CORE_OK;
    if ((rc = check_device())) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    ac::RopeArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.yq = static_cast<uint16_t*>(yq);
    a.yk = static_cast<uint16_t*>(yk);
    for (int i = 0; i < 3; ++i) {
        a.q_stride[i] = p->q_stride[i];
        a.k_stride[i] = p->k_stride[i];
        a.yq_stride[i] = p->yq_stride[i];
        a.yk_stride[i] = p->yk_stride[i];
    }
    a.s = p->s;
    a.h_q = p->h_q;
    a.h_kv = p->h_kv;
    a.pos0 = p->pos0;
    a.positions = p->positions;
    a.sign = sign;
    return ac::launch_rope(*reinterpret_cast<const ac::RopeTable*>(t), a, p->b, sms,
                           reinterpret_cast<cudaStream_t>(stream))
               ? ATTN_CORE_ERR_CUDA
               : ATTN_CORE_OK;
}

}  // namespace

extern "C" {

int attn_core_rope_init(const attn_core_rope_config* c, attn_core_rope_table* out)
{
    if (c == nullptr || out == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    const int32_t rot = c->rot_dim ? c->rot_dim : (c->d < 256 ? c->d : 256);
    attn_core_rope_table t{};
    t.d = c->d;
    t.rot_dim = rot;
    t.interleaved = c->interleaved;
    int rc = check_rope_table(&t);
    if (rc) return rc;
    const double base = c->base != 0.0 ? c->base : 10000.0;
    const double factor = c->factor != 0.0 ? c->factor : 1.0;
    const bool bands = c->low_freq != 0.0 || c->high_freq != 0.0;
    const double low = bands ? c->low_freq : 1.0, high = bands ? c->high_freq : 4.0;
    const bool betas = c->beta_fast != 0.0 || c->beta_slow != 0.0;
    const double fast = betas ? c->beta_fast : 32.0, slow = betas ? c->beta_slow : 1.0;
    const bool scaled = c->scaling != ATTN_CORE_ROPE_NONE;
    if (c->scaling < ATTN_CORE_ROPE_NONE || c->scaling > ATTN_CORE_ROPE_YARN || !positive(base) || base <= 1.0 ||
        !positive(factor) || (c->mscale != 0.0 && !positive(c->mscale)))
        return ATTN_CORE_ERR_INVALID_ARG;
    if ((c->scaling == ATTN_CORE_ROPE_BANDS || c->scaling == ATTN_CORE_ROPE_YARN) && !positive(c->original_len))
        return ATTN_CORE_ERR_INVALID_ARG;
    if (c->scaling == ATTN_CORE_ROPE_BANDS && !(low >= 0.0 && positive(high) && low < high))
        return ATTN_CORE_ERR_INVALID_ARG;
    if (c->scaling == ATTN_CORE_ROPE_YARN && !(positive(slow) && positive(fast) && slow < fast))
        return ATTN_CORE_ERR_INVALID_ARG;
    double lo = 0.0, hi = 0.0;
    if (c->scaling == ATTN_CORE_ROPE_YARN) {
        lo = floor(rot * log(c->original_len / (fast * kTwoPi)) / (2.0 * log(base)));
        hi = ceil(rot * log(c->original_len / (slow * kTwoPi)) / (2.0 * log(base)));
        lo = lo > 0.0 ? lo : 0.0;
        hi = hi < rot - 1 ? hi : rot - 1;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot);
        double keep = scaled ? 0.0 : 1.0;           // LINEAR slows every pair
        if (c->scaling == ATTN_CORE_ROPE_BANDS)
            keep = (c->original_len * f / kTwoPi - low) / (high - low);
        else if (c->scaling == ATTN_CORE_ROPE_YARN)
            keep = 1.0 - (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
        keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
        f = keep * f + (1.0 - keep) * (f / factor);
        // turns per position, whole turns dropped, as a 64-bit fraction
        const double turn = fmod(f / kTwoPi, 1.0);
        const double scaled_turn = ldexp(turn, 64);
        t.turns[i] = scaled_turn >= 18446744073709549568.0 ? ~(uint64_t)0 : (uint64_t)scaled_turn;
    }
    double m = c->mscale;
    if (m == 0.0) m = (c->scaling == ATTN_CORE_ROPE_YARN && factor > 1.0) ? 0.1 * log(factor) + 1.0 : 1.0;
    t.mscale = (float)m;
    *out = t;
    return ATTN_CORE_OK;
}

int attn_core_rope_fwd(const attn_core_rope_params* p, const attn_core_rope_table* t, const void* q, const void* k,
                       void* yq, void* yk, void* stream)
{
    return rope_call(p, t, q, k, yq, yk, 1.0f, stream);
}

int attn_core_rope_bwd(const attn_core_rope_params* p, const attn_core_rope_table* t, const void* dyq,
                       const void* dyk, void* dq, void* dk, void* stream)
{
    return rope_call(p, t, dyq, dyk, dq, dk, -1.0f, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The paged cache: append, attention, page copies.
namespace {

int check_paged(const attn_core_paged_params* p)
{
    if (p == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->n_seq <= 0 || p->n_tokens < 0 || p->h_q <= 0 || p->h_kv <= 0 || p->d <= 0 || p->n_pages <= 0 ||
        p->max_pages <= 0 || p->h_q % p->h_kv != 0)
        return ATTN_CORE_ERR_INVALID_ARG;
    if (!p->cu_seqlens_q || !p->kv_lens || !p->page_table) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->causal != 0 && p->causal != 1) return ATTN_CORE_ERR_INVALID_ARG;
    if (isnan(p->scale) || isinf(p->scale)) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->flags & ~ATTN_CORE_FLAG_TEST_WAIT_TIMEOUT) return ATTN_CORE_ERR_INVALID_ARG;
    const int ps = p->page_size;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!supported_d(p->d) || p->h_q / p->h_kv > kBlockRows || p->h_q + 2 * (int64_t)p->h_kv > kMaxHeads)
        return ATTN_CORE_ERR_UNSUPPORTED;
    // row counts that the kernels hold in 32 bits; element offsets are 64-bit
    if ((int64_t)p->n_pages * p->h_kv >= (int64_t)INT32_MAX ||
        (int64_t)p->max_pages * ps >= (int64_t)INT32_MAX - 2 * kBlockRows ||
        (int64_t)p->n_tokens * p->h_q >= (int64_t)INT32_MAX)
        return ATTN_CORE_ERR_INVALID_ARG;
    // the units of work of one KV head (paged_sched.cuh)
    const int64_t tpt = ac::paged_tokens_per_tile(p->h_q / p->h_kv);
    if ((p->n_tokens + tpt - 1) / tpt * (((int64_t)p->max_pages * ps + kBlockRows - 1) / kBlockRows) >=
        (int64_t)INT32_MAX || p->n_tokens >= INT32_MAX - 2 * kBlockRows)
        return ATTN_CORE_ERR_UNSUPPORTED;
    for (const void* t : {(const void*)p->cu_seqlens_q, (const void*)p->kv_lens, (const void*)p->page_table})
        if (reinterpret_cast<uintptr_t>(t) & 3u) return ATTN_CORE_ERR_MISALIGNED;
    return ATTN_CORE_OK;
}

ac::PagedTables paged_tables(const attn_core_paged_params* p)
{
    ac::PagedTables t{};
    t.cu_q = p->cu_seqlens_q;
    t.kv_lens = p->kv_lens;
    t.page_table = p->page_table;
    t.n_seq = p->n_seq;
    t.n_tokens = p->n_tokens;
    t.h_q = p->h_q;
    t.h_kv = p->h_kv;
    t.page_size = p->page_size;
    for (t.page_shift = 0; (1 << t.page_shift) < p->page_size;) ++t.page_shift;
    t.n_pages = p->n_pages;
    t.max_pages = p->max_pages;
    t.status = p->dev_status;
    return t;
}

int compare_ints(const void* a, const void* b)
{
    const int32_t x = *static_cast<const int32_t*>(a), y = *static_cast<const int32_t*>(b);
    return x < y ? -1 : x > y;
}

// Every page in range, every target named once and no target a source.
int check_pairs(const int32_t* pairs, int64_t n, int64_t n_pages)
{
    for (int64_t i = 0; i < 2 * n; ++i)
        if (pairs[i] < 0 || pairs[i] >= n_pages) return ATTN_CORE_ERR_INVALID_ARG;
    if (n > n_pages) return ATTN_CORE_ERR_INVALID_ARG;
    if (n <= 16) {
        for (int64_t i = 0; i < n; ++i)
            for (int64_t j = 0; j < n; ++j)
                if (pairs[2 * i + 1] == pairs[2 * j] || (i != j && pairs[2 * i + 1] == pairs[2 * j + 1]))
                    return ATTN_CORE_ERR_INVALID_ARG;
        return ATTN_CORE_OK;
    }
    int32_t* dst = static_cast<int32_t*>(malloc((size_t)n * sizeof(int32_t)));
    if (dst == nullptr) return ATTN_CORE_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i) dst[i] = pairs[2 * i + 1];
    qsort(dst, (size_t)n, sizeof(int32_t), compare_ints);
    int rc = ATTN_CORE_OK;
    for (int64_t i = 1; i < n && !rc; ++i)
        if (dst[i] == dst[i - 1]) rc = ATTN_CORE_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n && !rc; ++i)
        if (bsearch(&pairs[2 * i], dst, (size_t)n, sizeof(int32_t), compare_ints)) rc = ATTN_CORE_ERR_INVALID_ARG;
    free(dst);
    return rc;
}

}  // namespace

extern "C" {

int attn_core_paged_append(const attn_core_paged_params* p, const attn_core_rope_table* t, const void* q,
                           const void* k, const void* v, const int64_t* strides, void* q_out, void* k_pages,
                           void* v_pages, void* stream)
{
    int rc = check_paged(p);
    if (rc) return rc;
    if (!k || !v || !k_pages || !v_pages || (q == nullptr) != (q_out == nullptr)) return ATTN_CORE_ERR_INVALID_ARG;
    if (p->flags) return ATTN_CORE_ERR_INVALID_ARG;   // no wait in this kernel to time out
    if (t != nullptr) {
        if ((rc = check_rope_table(t))) return rc;
        if (t->d != p->d) return ATTN_CORE_ERR_INVALID_ARG;
    }
    const int64_t packed[3] = {(int64_t)p->h_q * p->d, (int64_t)p->h_kv * p->d, (int64_t)p->h_kv * p->d};
    for (int i = 0; i < 3 && strides; ++i) {
        if (i == 0 && !q) continue;
        if (strides[i] < 0 || strides[i] > ((int64_t)1 << 42)) return ATTN_CORE_ERR_INVALID_ARG;
        if (strides[i] % 8) return ATTN_CORE_ERR_MISALIGNED;
    }
    if (!strides) strides = packed;
    if (q && q == q_out && strides[0] != packed[0]) return ATTN_CORE_ERR_INVALID_ARG;
    if (k_pages == v_pages || (q_out && (q_out == k || q_out == v || q_out == k_pages || q_out == v_pages)))
        return ATTN_CORE_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, (const void*)q_out, (const void*)k_pages, (const void*)v_pages})
        if (!aligned16(x)) return ATTN_CORE_ERR_MISALIGNED;
    if (p->n_tokens == 0) return ATTN_CORE_OK;
    if ((rc = check_device())) return rc;
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    ac::AppendArgs a{};
    a.t = paged_tables(p);
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q ? strides[0] : 0;
    a.k_stride = strides[1];
    a.v_stride = strides[2];
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_pages = static_cast<uint16_t*>(k_pages);
    a.v_pages = static_cast<uint16_t*>(v_pages);
    ac::RopeTable none{};            // no rotation: every unit is a copy
    none.d = p->d;
    none.mscale = 1.0f;
    const ac::RopeTable& rt = t ? *reinterpret_cast<const ac::RopeTable*>(t) : none;
    return ac::launch_append(rt, a, sms, reinterpret_cast<cudaStream_t>(stream)) ? ATTN_CORE_ERR_CUDA : ATTN_CORE_OK;
}

size_t attn_core_paged_workspace_bytes(const attn_core_paged_params* p)
{
    return check_paged(p) ? 0 : ac::paged_ws_bytes(p->d);
}

int attn_core_paged_fwd(const attn_core_paged_params* p, const void* q, const void* k_pages, const void* v_pages,
                        void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_paged(p);
    if (rc) return rc;
    if (!q || !k_pages || !v_pages || !o || !lse || !workspace) return ATTN_CORE_ERR_INVALID_ARG;
    if (o == q || o == k_pages || o == v_pages) return ATTN_CORE_ERR_INVALID_ARG;
    for (const void* x : {q, k_pages, v_pages, (const void*)o, (const void*)lse})
        if (!aligned16(x)) return ATTN_CORE_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return ATTN_CORE_ERR_MISALIGNED;
    if (workspace_bytes < ac::paged_ws_bytes(p->d)) return ATTN_CORE_ERR_WORKSPACE_TOO_SMALL;
    if (p->n_tokens == 0) return ATTN_CORE_OK;
    if ((rc = check_device())) return rc;
    if ((rc = get_encoder())) return rc;
    ac::PagedArgs a{};
    a.t = paged_tables(p);
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(workspace);
    a.d = p->d;
    a.causal = p->causal;
    a.group = p->h_q / p->h_kv;
    a.tpt = ac::paged_tokens_per_tile(a.group);
    const float scale = (p->scale > 0.0f) ? p->scale : 1.0f / sqrtf((float)p->d);
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.timeout_ns = (uint64_t)(p->wait_timeout_ms ? p->wait_timeout_ms : 2000u) * 1000000ull;
    a.inject_timeout = (p->flags & ATTN_CORE_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    if ((rc = device_sms(&a.num_sms))) return rc;
    ac::PagedMaps m;
    for (int i = 0; i < (p->d % 64 ? 2 : 1); ++i) {
        const int cw = i ? 32 : 64;
        const int64_t pages = (int64_t)p->n_pages * p->h_kv;
        if ((rc = encode_map_tokens(&m.q[i], q, cw, p->d, a.group, p->h_kv, p->n_tokens, a.tpt)) ||
            (rc = encode_map_pages(&m.k[i], k_pages, cw, p->d, p->page_size, pages)) ||
            (rc = encode_map_pages(&m.v[i], v_pages, cw, p->d, p->page_size, pages)))
            return rc;
    }
    if ((rc = encode_map_tokens(&m.o, o, p->d % 64 ? 32 : 64, p->d, a.group, p->h_kv, p->n_tokens, a.tpt))) return rc;
    return ac::launch_paged(m, a, reinterpret_cast<cudaStream_t>(stream)) ? ATTN_CORE_ERR_CUDA : ATTN_CORE_OK;
}

int attn_core_page_copy(void* pages, int64_t n_planes, int64_t plane_stride, int64_t n_pages, int64_t page_bytes,
                        const int32_t* pairs, int64_t n_pairs, void* stream)
{
    if (!pages || n_planes <= 0 || n_pages <= 0 || n_pages > (int64_t)INT32_MAX || page_bytes <= 0 || n_pairs < 0 ||
        (n_pairs > 0 && !pairs))
        return ATTN_CORE_ERR_INVALID_ARG;
    // sizes whose products stay in range (65535: blocks in y; 2 GiB a page)
    if (n_planes > 65535 || page_bytes > ((int64_t)1 << 31)) return ATTN_CORE_ERR_UNSUPPORTED;
    if (!aligned16(pages) || page_bytes % 16 || plane_stride % 16) return ATTN_CORE_ERR_MISALIGNED;
    if (n_planes > 1 && plane_stride < n_pages * page_bytes) return ATTN_CORE_ERR_INVALID_ARG;
    int rc = check_pairs(pairs, n_pairs, n_pages);
    if (rc) return rc;
    if (n_pairs == 0) return ATTN_CORE_OK;
    if ((rc = check_device())) return rc;
    return ac::launch_page_copy(pages, n_planes, plane_stride, page_bytes, pairs, n_pairs,
                                reinterpret_cast<cudaStream_t>(stream))
               ? ATTN_CORE_ERR_CUDA
               : ATTN_CORE_OK;
}

}  // extern "C"
