// C ABI of the attention half (moedec_attn.h): argument validation and launches.
// Every entry point checks its arguments on the host before anything is
// enqueued.
#include <math.h>

#include "attn.h"

#define MOEDEC_API extern "C" __attribute__((visibility("default")))

using namespace moedec::attn;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dtype_ok(int d) { return d == MOEDEC_F32 || d == MOEDEC_F16 || d == MOEDEC_BF16; }
int64_t dtype_bytes(int d) { return d == MOEDEC_F32 ? 4 : 2; }
int status(hipError_t e) { return e == hipSuccess ? MOEDEC_OK : MOEDEC_ERR_DEVICE; }

constexpr int64_t kMaxRows = 1 << 24;
constexpr int64_t kMaxGrid = 0x7FFFFFFF;

// Checks the cache and fills `out`.
int check_cache(const kv4_cache* c, Cache& out) {
    if (!c || !c->data || !c->table || !c->len || !c->ref) return MOEDEC_ERR_INVALID_ARG;
    if (c->layers < 1 || c->n_pages < 1 || c->page_tokens < 1 || c->kv_heads < 1 || c->head_dim < 1 ||
        c->n_seqs < 1 || c->max_pages < 1)
        return MOEDEC_ERR_INVALID_ARG;
    if (!aligned16(c->data) || !aligned16(c->ref) || !aligned4(c->table) || !aligned4(c->len))
        return MOEDEC_ERR_INVALID_ARG;
    const int pt = c->page_tokens;
    if ((pt != 32 && pt != 64 && pt != 128) ||
        (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256) ||
        c->kv_heads > 1024 || c->n_seqs > KV4_MAX_SEQS || c->n_pages > (1 << 24) ||
        (int64_t)c->max_pages * pt > (1 << 30))
        return MOEDEC_ERR_UNSUPPORTED;
    out.data = c->data;
    out.table = c->table;
    out.len = c->len;
    out.ref = c->ref;
    out.layers = c->layers;
    out.n_pages = c->n_pages;
    out.kv_heads = c->kv_heads;
    out.n_seqs = c->n_seqs;
    out.max_pages = c->max_pages;
    out.pt_log2 = pt == 32 ? 5 : pt == 64 ? 6 : 7;
    out.head_dim = c->head_dim;
    return MOEDEC_OK;
}

bool stride_ok(int64_t ld, int64_t row, int dtype) { return ld >= row && ld * dtype_bytes(dtype) % 16 == 0; }

// Whether rows of wa elements lda apart and rows of wb elements ldb apart share an
// element.  Rows of one stride may interleave (columns of one buffer); others
// count as shared where their ranges meet.
bool overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t rows,
             int64_t bytes) {
    const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a), pb = (int64_t)reinterpret_cast<uintptr_t>(b);
    if (pa + ((rows - 1) * lda + wa) * bytes <= pb || pb + ((rows - 1) * ldb + wb) * bytes <= pa) return false;
    if (rows == 1 || lda != ldb) return true;
    const int64_t ld = lda * bytes, d = ((pb - pa) % ld + ld) % ld;
    return d < wa * bytes || d + wb * bytes > ld;
}

int check_rows(const Cache& c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
               int64_t rows, const int32_t* q_start) {
    if (!q_start || !aligned4(q_start) || layer < 0 || layer >= c.layers || rows < 0 || !dtype_ok(dtype))
        return MOEDEC_ERR_INVALID_ARG;
    if (rows > 0 && (!k || !v)) return MOEDEC_ERR_INVALID_ARG;
    const int64_t row = (int64_t)c.kv_heads * c.head_dim;
    if (!stride_ok(ldk, row, dtype) || !stride_ok(ldv, row, dtype) || !aligned16(k) || !aligned16(v))
        return MOEDEC_ERR_INVALID_ARG;
    if (rows >= kMaxRows || (rows / 8 + 2 * c.n_seqs) * (int64_t)c.kv_heads * 2 > kMaxGrid)
        return MOEDEC_ERR_UNSUPPORTED;
    return MOEDEC_OK;
}

int check_attention(const Cache& c, int64_t rows, int heads, int64_t max_len) {
    if (rows < 0 || heads < 1 || heads % c.kv_heads || max_len < 1) return MOEDEC_ERR_INVALID_ARG;
    if (rows >= kMaxRows || heads > 16384 || attention_grid(c, (int)rows, heads, max_len) > kMaxGrid)
        return MOEDEC_ERR_UNSUPPORTED;
    return MOEDEC_OK;
}

int linear(int bits, const void* x, int dtype, int64_t ldx, const uint8_t* w, const float* scale, const float* bias,
           int act, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t K, int64_t N,
           void* workspace, int64_t workspace_bytes, void* stream) {
    if (T < 0 || K < 1 || N < 1 || !dtype_ok(dtype) || act < MOEDEC_ACT_NONE || act > MOEDEC_ACT_RELU)
        return MOEDEC_ERR_INVALID_ARG;
    if (!w || !scale || K % (128 / bits) || !aligned16(w) || !aligned4(scale) || !aligned4(bias))
        return MOEDEC_ERR_INVALID_ARG;
    if (T == 0) return MOEDEC_OK;
    if (!x || !y || !aligned16(x) || !stride_ok(ldx, K, dtype) || ldy < N || (residual && ldr < N))
        return MOEDEC_ERR_INVALID_ARG;
    const uintptr_t e = (uintptr_t)dtype_bytes(dtype) - 1;
    if ((reinterpret_cast<uintptr_t>(y) & e) || (reinterpret_cast<uintptr_t>(residual) & e))
        return MOEDEC_ERR_INVALID_ARG;
    if (K > 65536 || T >= kMaxRows || N >= kMaxRows) return MOEDEC_ERR_UNSUPPORTED;
    const int64_t bytes = dtype_bytes(dtype);
    if (overlap(x, ldx, K, y, ldy, N, T, bytes)) return MOEDEC_ERR_INVALID_ARG;
    if (residual && (residual != y || (ldr != ldy && T > 1)) && overlap(residual, ldr, N, y, ldy, N, T, bytes))
        return MOEDEC_ERR_INVALID_ARG;
    const int64_t need = linear_workspace(bits, dtype, T, K, N);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return MOEDEC_ERR_INVALID_ARG;
    LinearArgs a;
    a.x = x;
    a.w = w;
    a.scale = scale;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.workspace = workspace;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.T = (int)T;
    a.K = (int)K;
    a.N = (int)N;
    a.act = act;
    if (linear_grid(a) > kMaxGrid) return MOEDEC_ERR_UNSUPPORTED;
    return status(launch_linear(bits, dtype, a, static_cast<hipStream_t>(stream)));
}

}  // namespace

MOEDEC_API int64_t dense_linear_workspace(int bits, int dtype, int64_t T, int64_t K, int64_t N) {
    if ((bits != 4 && bits != 8 && bits != 2) || !dtype_ok(dtype) || T < 0 || K < 1 || N < 1 || K > 65536 ||
        T >= kMaxRows || N >= kMaxRows)
        return -1;
    return linear_workspace(bits, dtype, T, K, N);
}

#define DENSE_LINEAR(BITS)                                                                                            \
    MOEDEC_API int dense_linear_q##BITS(const void* x, int dtype, int64_t ldx, const uint8_t* w, const float* scale,  \
                                        const float* bias, int act, const void* residual, int64_t ldr, void* y,       \
                                        int64_t ldy, int64_t T, int64_t K, int64_t N, void* workspace,                \
                                        int64_t workspace_bytes, void* stream) {                                      \
        return linear(BITS, x, dtype, ldx, w, scale, bias, act, residual, ldr, y, ldy, T, K, N, workspace,            \
                      workspace_bytes, stream);                                                                       \
    }
DENSE_LINEAR(4)
DENSE_LINEAR(8)
DENSE_LINEAR(2)

MOEDEC_API int kv4_append(const kv4_cache* cache, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv,
                          int dtype, int64_t rows, const int32_t* q_start, const int32_t* granted, void* stream) {
    Cache c;
    int st = check_cache(cache, c);
    if (st == MOEDEC_OK) st = check_rows(c, layer, k, ldk, v, ldv, dtype, rows, q_start);
    if (st != MOEDEC_OK) return st;
    if (!aligned4(granted)) return MOEDEC_ERR_INVALID_ARG;
    return status(launch_append(c, layer, k, ldk, v, ldv, dtype, (int)rows, q_start, granted,
                                static_cast<hipStream_t>(stream)));
}

MOEDEC_API int kv4_read(const kv4_cache* cache, int layer, const int32_t* first, const int32_t* q_start, int64_t rows,
                        void* k, int64_t ldk, void* v, int64_t ldv, int dtype, void* stream) {
    Cache c;
    int st = check_cache(cache, c);
    if (st == MOEDEC_OK) st = check_rows(c, layer, k, ldk, v, ldv, dtype, rows, q_start);
    if (st != MOEDEC_OK) return st;
    if (!first || !aligned4(first)) return MOEDEC_ERR_INVALID_ARG;
    return status(launch_read(c, layer, first, q_start, (int)rows, k, ldk, v, ldv, dtype,
                              static_cast<hipStream_t>(stream)));
}

MOEDEC_API int64_t kv4_attention_workspace(const kv4_cache* cache, int64_t rows, int heads, int64_t max_len) {
    Cache c;
    if (check_cache(cache, c) != MOEDEC_OK || check_attention(c, rows, heads, max_len) != MOEDEC_OK) return -1;
    return attention_workspace(c, (int)rows, heads, max_len);
}

MOEDEC_API int kv4_attention(const kv4_cache* cache, int layer, const void* q, int64_t ldq, int dtype, int64_t rows,
                             int heads, const int32_t* q_start, const int32_t* granted, float scale, int window,
                             int64_t max_len, void* out, int64_t ldo, float* lse, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    Cache c;
    int st = check_cache(cache, c);
    if (st == MOEDEC_OK) st = check_attention(c, rows, heads, max_len);
    if (st != MOEDEC_OK) return st;
    if (!q_start || !aligned4(q_start) || !aligned4(granted) || !aligned4(lse) || layer < 0 || layer >= c.layers ||
        !dtype_ok(dtype) || !isfinite(scale) || window < 0)
        return MOEDEC_ERR_INVALID_ARG;
    if (rows == 0) return MOEDEC_OK;
    const int64_t row = (int64_t)heads * c.head_dim;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !stride_ok(ldq, row, dtype) || !stride_ok(ldo, row, dtype))
        return MOEDEC_ERR_INVALID_ARG;
    if (overlap(q, ldq, row, out, ldo, row, rows, dtype_bytes(dtype))) return MOEDEC_ERR_INVALID_ARG;
    const int64_t need = attention_workspace(c, (int)rows, heads, max_len);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return MOEDEC_ERR_INVALID_ARG;
    AttnArgs a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_start = q_start;
    a.granted = granted;
    a.workspace = workspace;
    a.ldq = ldq;
    a.ldo = ldo;
    a.layer = layer;
    a.rows = (int)rows;
    a.heads = heads;
    a.window = window;
    a.scale = scale;
    a.max_len = max_len;
    return status(launch_attention(c, a, dtype, static_cast<hipStream_t>(stream)));
}

MOEDEC_API int kv4_reserve(const kv4_cache* cache, const int32_t* n_new, int32_t* granted, int32_t* workspace,
                           void* stream) {
    Cache c;
    const int st = check_cache(cache, c);
    if (st != MOEDEC_OK) return st;
    if (!n_new || !granted || !workspace || !aligned4(n_new) || !aligned4(granted) || !aligned4(workspace))
        return MOEDEC_ERR_INVALID_ARG;
    return status(launch_reserve(c, n_new, granted, workspace, static_cast<hipStream_t>(stream)));
}

MOEDEC_API int kv4_fork(const kv4_cache* cache, int n, const int32_t* src, const int32_t* dst,
                        const int32_t* n_tokens, int32_t* ok, void* stream) {
    Cache c;
    const int st = check_cache(cache, c);
    if (st != MOEDEC_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst || !ok)) || !aligned4(src) || !aligned4(dst) || !aligned4(n_tokens) ||
        !aligned4(ok))
        return MOEDEC_ERR_INVALID_ARG;
    if (n > KV4_MAX_SEQS) return MOEDEC_ERR_UNSUPPORTED;
    return status(launch_fork(c, n, src, dst, n_tokens, ok, static_cast<hipStream_t>(stream)));
}

MOEDEC_API int kv4_truncate(const kv4_cache* cache, const int32_t* new_len, void* stream) {
    Cache c;
    const int st = check_cache(cache, c);
    if (st != MOEDEC_OK) return st;
    if (!new_len || !aligned4(new_len)) return MOEDEC_ERR_INVALID_ARG;
    return status(launch_truncate(c, new_len, static_cast<hipStream_t>(stream)));
}

MOEDEC_API int kv4_compact(const kv4_cache* cache, int32_t* remap, int32_t* n_live, int32_t* workspace,
                           void* stream) {
    Cache c;
    const int st = check_cache(cache, c);
    if (st != MOEDEC_OK) return st;
    if (!remap || !n_live || !workspace || !aligned4(remap) || !aligned4(n_live) || !aligned4(workspace))
        return MOEDEC_ERR_INVALID_ARG;
    return status(launch_compact(c, remap, n_live, workspace, static_cast<hipStream_t>(stream)));
}
