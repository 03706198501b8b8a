// Host side of the paged 4-bit cache (include/moba.h): argument checks, workspace layout, launches.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "cache_internal.cuh"
#include "moba.h"

using namespace moba;

namespace moba {
void set_error_message(const char* msg);
}

namespace {

struct NvtxScope {
    explicit NvtxScope(const char* name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
    NvtxScope(const NvtxScope&) = delete;
    NvtxScope& operator=(const NvtxScope&) = delete;
};

moba_status fail(moba_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moba_status fail(moba_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_error_message(buf);
    return s;
}

moba_status cuda_fail(cudaError_t e, const char* what) {
    return fail(MOBA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

// The sizes of a cache, without its buffers.
moba_status check_shape(const moba_cache* c) {
    if (!c) return fail(MOBA_ERR_INVALID_ARG, "cache is NULL");
    if (c->num_pages < 1 || c->num_seqs < 1 || c->max_blocks < 1 || c->num_kv_heads < 1 || c->head_dim < 1 ||
        c->chunk_size < 1)
        return fail(MOBA_ERR_INVALID_ARG, "cache sizes must be >= 1 (pages %d, sequences %d, blocks %d, heads %d, "
                    "head_dim %d, chunk %d)", c->num_pages, c->num_seqs, c->max_blocks, c->num_kv_heads,
                    c->head_dim, c->chunk_size);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(MOBA_ERR_UNSUPPORTED, "head_dim %d unsupported (64 or 128)", c->head_dim);
    if (c->chunk_size % 128 || c->chunk_size > (1 << 20))
        return fail(MOBA_ERR_UNSUPPORTED, "chunk_size %d unsupported (multiple of 128, <= 2^20)", c->chunk_size);
    if (c->num_seqs > 65535 || c->num_kv_heads > 65535)
        return fail(MOBA_ERR_UNSUPPORTED, "num_seqs %d or num_kv_heads %d unsupported (<= 65535)", c->num_seqs,
                    c->num_kv_heads);
    if ((long long)c->max_blocks * c->chunk_size > 0x7fffffffLL)
        return fail(MOBA_ERR_UNSUPPORTED, "max_blocks %d * chunk_size %d exceeds 2^31 - 1", c->max_blocks,
                    c->chunk_size);
    if (c->num_pages > 0x7fff0000)
        return fail(MOBA_ERR_UNSUPPORTED, "num_pages %d unsupported", c->num_pages);
    if (c->k_exp < -64 || c->k_exp > 64 || c->v_exp < -64 || c->v_exp > 64)
        return fail(MOBA_ERR_UNSUPPORTED, "k_exp %d or v_exp %d unsupported (-64..64)", c->k_exp, c->v_exp);
    return MOBA_OK;
}

moba_status check_cache(const moba_cache* c) {
    const moba_status s = check_shape(c);
    if (s != MOBA_OK) return s;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->k_mean || !c->table || !c->lengths ||
        !c->refs || !c->status)
        return fail(MOBA_ERR_INVALID_ARG, "NULL buffer in the cache");
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
        !aligned(c->v_scales, 16) || !aligned(c->k_mean, 16))
        return fail(MOBA_ERR_INVALID_ARG, "the cache's pools and k_mean must be 16-byte aligned");
    if (!aligned(c->table, 4) || !aligned(c->lengths, 4) || !aligned(c->refs, 4) || !aligned(c->status, 4))
        return fail(MOBA_ERR_INVALID_ARG, "the cache's int32 buffers must be 4-byte aligned");
    return MOBA_OK;
}

moba_status check_workspace(const void* ws, size_t bytes, size_t need) {
    if (!ws || bytes < need)
        return fail(MOBA_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws ? bytes : (size_t)0);
    if (!aligned(ws, 256)) return fail(MOBA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return MOBA_OK;
}

cache::View view(const moba_cache& c) {
    cache::View v;
    v.pages = c.num_pages;
    v.seqs = c.num_seqs;
    v.max_blocks = c.max_blocks;
    v.hkv = c.num_kv_heads;
    v.d = c.head_dim;
    v.chunk = c.chunk_size;
    v.k_unit = ldexpf(1.f, c.k_exp);
    v.v_unit = ldexpf(1.f, c.v_exp);
    v.kc = static_cast<uint8_t*>(c.k_codes);
    v.ks = static_cast<uint8_t*>(c.k_scales);
    v.vc = static_cast<uint8_t*>(c.v_codes);
    v.vs = static_cast<uint8_t*>(c.v_scales);
    v.mean = c.k_mean;
    v.table = c.table;
    v.lengths = c.lengths;
    v.refs = c.refs;
    v.status = c.status;
    return v;
}

// Multiprocessors of the current device, asked for once per device.
int device_sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

size_t page_ws_bytes(const moba_cache& c) { return 4 * cache::page_ws_words(c.num_pages, c.num_seqs); }

struct DecodeLayout {
    int hgroups, rows, row_heads, max_items;
    size_t items, tiles, done, part_o, part_ml, total;
};

// Shapes of a decode call; MOBA_OK with the layout in *L.
moba_status decode_layout(const moba_cache* c, int hq, int topk, DecodeLayout* L) {
    const moba_status s = check_shape(c);
    if (s != MOBA_OK) return s;
    if (hq < 1 || hq % c->num_kv_heads)
        return fail(MOBA_ERR_INVALID_ARG, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)", hq,
                    c->num_kv_heads);
    if (topk < 0) return fail(MOBA_ERR_INVALID_ARG, "topk must be >= 0 (got %d)", topk);
    if (topk > 32) return fail(MOBA_ERR_UNSUPPORTED, "topk %d unsupported (<= 32, or 0 for every block)", topk);
    const int group = hq / c->num_kv_heads;
    L->hgroups = (group + cache::kRowHeads - 1) / cache::kRowHeads;
    const long long rows = (long long)c->num_seqs * c->num_kv_heads * L->hgroups;
    if (rows > (1LL << 24))
        return fail(MOBA_ERR_UNSUPPORTED, "num_seqs * num_q_heads too large (%lld rows of heads)", rows);
    // the attention counts the tiles of all rows in 32 bits
    if (rows * (((long long)c->max_blocks * c->chunk_size + 63) / 64) > 0x7fffffffLL)
        return fail(MOBA_ERR_UNSUPPORTED, "num_seqs * query head groups * max_blocks * chunk_size / 64 exceeds 2^31");
    L->rows = (int)rows;
    L->row_heads = group < cache::kRowHeads ? group : cache::kRowHeads;
    const int most = L->row_heads * (topk - 1) + 1;
    L->max_items = topk == 0 ? 0 : most < c->max_blocks ? most : c->max_blocks;
    L->items = 0;
    L->tiles = align_up(sizeof(int2) * (size_t)L->rows * L->max_items);
    L->done = L->tiles + align_up(4ull * L->rows);
    L->part_o = L->done + align_up(4ull * L->rows);
    const size_t parts = cache::most_parts(L->rows);
    L->part_ml = L->part_o + align_up(4 * parts * L->row_heads * c->head_dim);
    L->total = L->part_ml + align_up(sizeof(float2) * parts * L->row_heads);
    return MOBA_OK;
}

}  // namespace

extern "C" {

size_t moba_cache_workspace_size(const moba_cache* c) {
    if (check_shape(c) != MOBA_OK) return 0;
    return page_ws_bytes(*c);
}

moba_status moba_cache_reserve(const moba_cache* c, const int* upto, void* workspace, size_t workspace_bytes,
                               void* stream) {
    NvtxScope range("moba_cache_reserve");
    moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    if (!upto) return fail(MOBA_ERR_INVALID_ARG, "NULL pointer argument");
    s = check_workspace(workspace, workspace_bytes, page_ws_bytes(*c));
    if (s != MOBA_OK) return s;
    const cudaError_t e = cache::launch_reserve(view(*c), upto, static_cast<int*>(workspace),
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache reserve launch");
}

moba_status moba_cache_append(const moba_cache* c, const void* k, const void* v, const int* cu_new,
                              const int* start, int new_tokens, void* k_held, void* v_held, void* stream) {
    NvtxScope range("moba_cache_append");
    const moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    if (new_tokens < 0) return fail(MOBA_ERR_INVALID_ARG, "new_tokens must be >= 0 (got %d)", new_tokens);
    if (new_tokens == 0) return MOBA_OK;
    if (!k || !v || !cu_new || !start) return fail(MOBA_ERR_INVALID_ARG, "NULL pointer argument");
    if (!k_held != !v_held) return fail(MOBA_ERR_INVALID_ARG, "k_held and v_held go together");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_held, 16) || !aligned(v_held, 16))
        return fail(MOBA_ERR_INVALID_ARG, "k, v, k_held and v_held must be 16-byte aligned");
    cache::AppendArgs a;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.cu = cu_new;
    a.start = start;
    a.total = new_tokens;
    a.k_held = static_cast<__nv_bfloat16*>(k_held);
    a.v_held = static_cast<__nv_bfloat16*>(v_held);
    const cudaError_t e = cache::launch_append(view(*c), a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache append launch");
}

size_t moba_cache_decode_workspace_size(const moba_cache* c, int num_q_heads, int topk) {
    DecodeLayout L;
    return decode_layout(c, num_q_heads, topk, &L) == MOBA_OK ? L.total : 0;
}

moba_status moba_cache_decode(const moba_cache* c, const void* q, int num_q_heads, int topk,
                              float softmax_scale, void* workspace, size_t workspace_bytes, void* out,
                              float* lse, void* stream) {
    NvtxScope range("moba_cache_decode");
    DecodeLayout L;
    moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    s = decode_layout(c, num_q_heads, topk, &L);
    if (s != MOBA_OK) return s;
    if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale))
        return fail(MOBA_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (!q || !out || !lse) return fail(MOBA_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
        return fail(MOBA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    s = check_workspace(workspace, workspace_bytes, L.total);
    if (s != MOBA_OK) return s;
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)c->head_dim);
    const float scale_log2 = ldexpf(scale * 1.4426950408889634f, c->k_exp);
    if (std::isinf(scale_log2))
        return fail(MOBA_ERR_INVALID_ARG, "softmax_scale %g with k_exp %d passes the range of fp32", softmax_scale, c->k_exp);
    cache::DecodeArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.hq = num_q_heads;
    a.group = num_q_heads / c->num_kv_heads;
    a.topk = topk;
    a.hgroups = L.hgroups;
    a.rows = L.rows;
    a.row_heads = L.row_heads;
    a.max_items = L.max_items;
    a.scale_log2 = scale_log2;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    cache::DecodeWs ws;
    char* base = static_cast<char*>(workspace);
    ws.items = reinterpret_cast<int2*>(base + L.items);
    ws.tiles = reinterpret_cast<int*>(base + L.tiles);
    ws.done = reinterpret_cast<int*>(base + L.done);
    ws.part_o = reinterpret_cast<float*>(base + L.part_o);
    ws.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
    const cudaError_t e = cache::launch_decode(view(*c), a, ws, device_sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache decode launch");
}

moba_status moba_cache_fork(const moba_cache* c, const int* src, const int* dst, int n, void* workspace,
                            size_t workspace_bytes, void* stream) {
    NvtxScope range("moba_cache_fork");
    moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    if (n < 0 || n > c->num_seqs)
        return fail(MOBA_ERR_INVALID_ARG, "n must be in 0..num_seqs (got %d)", n);
    if (n == 0) return MOBA_OK;
    if (!src || !dst) return fail(MOBA_ERR_INVALID_ARG, "NULL pointer argument");
    s = check_workspace(workspace, workspace_bytes, page_ws_bytes(*c));
    if (s != MOBA_OK) return s;
    const cudaError_t e = cache::launch_fork(view(*c), src, dst, n, static_cast<int*>(workspace),
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache fork launch");
}

moba_status moba_cache_free(const moba_cache* c, const int* seqs, int n, void* stream) {
    NvtxScope range("moba_cache_free");
    const moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    if (n < 0) return fail(MOBA_ERR_INVALID_ARG, "n must be >= 0 (got %d)", n);
    if (n == 0) return MOBA_OK;
    if (!seqs) return fail(MOBA_ERR_INVALID_ARG, "NULL pointer argument");
    const cudaError_t e = cache::launch_free(view(*c), seqs, n, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache free launch");
}

moba_status moba_cache_compact(const moba_cache* c, const moba_cache* into, void* workspace,
                               size_t workspace_bytes, void* stream) {
    NvtxScope range("moba_cache_compact");
    moba_status s = check_cache(c);
    if (s == MOBA_OK) s = check_cache(into);
    if (s != MOBA_OK) return s;
    if (c->num_kv_heads != into->num_kv_heads || c->head_dim != into->head_dim ||
        c->chunk_size != into->chunk_size || c->k_exp != into->k_exp || c->v_exp != into->v_exp ||
        c->num_seqs != into->num_seqs || c->max_blocks != into->max_blocks)
        return fail(MOBA_ERR_INVALID_ARG, "compact: the caches differ in more than num_pages");
    if (c->k_codes == into->k_codes || c->k_scales == into->k_scales || c->v_codes == into->v_codes ||
        c->v_scales == into->v_scales || c->k_mean == into->k_mean || c->table == into->table ||
        c->lengths == into->lengths || c->refs == into->refs)
        return fail(MOBA_ERR_INVALID_ARG, "compact: the caches have a buffer in common");
    s = check_workspace(workspace, workspace_bytes, page_ws_bytes(*c));
    if (s != MOBA_OK) return s;
    const cudaError_t e = cache::launch_compact(view(*c), view(*into), static_cast<int*>(workspace),
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOBA_OK : cuda_fail(e, "cache compact launch");
}

moba_status moba_cache_status(const moba_cache* c, void* stream) {
    NvtxScope range("moba_cache_status");
    const moba_status s = check_cache(c);
    if (s != MOBA_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int code = 0;
    cudaError_t e = cudaMemcpyAsync(&code, c->status, sizeof(int), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && code) e = cudaMemsetAsync(c->status, 0, sizeof(int), st);
    if (e != cudaSuccess) return cuda_fail(e, "cache status read");
    switch (code) {
        case MOBA_OK: return MOBA_OK;
        case MOBA_ERR_INVALID_ARG:
            return fail(MOBA_ERR_INVALID_ARG, "a call on the cache met an index, length or page that does not fit");
        case MOBA_ERR_NO_PAGES: return fail(MOBA_ERR_NO_PAGES, "the cache has too few free pages");
        case MOBA_ERR_DEVICE_TIMEOUT: return fail(MOBA_ERR_DEVICE_TIMEOUT, "a bounded device wait gave up");
    }
    return fail(MOBA_ERR_INVALID_ARG, "the cache's status word holds %d", code);
}

}  // extern "C"
