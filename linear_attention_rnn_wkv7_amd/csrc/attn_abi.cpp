// C ABI of softmax attention, the norm and rotation before it and the paged
// cache: argument validation, workspace layout and dispatch.  Every check runs
// before anything is enqueued on the stream.

#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "attn_internal.h"
#include "wkv7_internal.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = int64_t(1) << 30;    // of a row, or of a row's pages
constexpr int64_t kMaxStride = int64_t(1) << 22;    // elements
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;   // of 256 threads: below 2^32

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, uintptr_t to = 16) { return (uintptr_t)p % to == 0; }
int status(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP; }
bool is_dtype(int32_t d) { return d == WKV7_F32 || d == WKV7_BF16; }
// (times log2 e it is still finite)
bool is_scale(float s) { return std::isnormal(s) && s > 0.f && s <= 0x1p127f; }
bool is_cache(int32_t d) { return d == KV_CACHE_SAME || d == KV_CACHE_E4M3; }

int check_workspace(const void *ws, size_t given, size_t need)
{
    if (need == 0) return WKV7_OK;
    return ws && given >= need && aligned(ws, kAlign) ? WKV7_OK : WKV7_ERR_WORKSPACE;
}

// The stride to use for `heads` heads of D, and whether `tokens` of it fit.
int check_stride(int64_t given, int64_t heads, int64_t D, int64_t tokens, int64_t *stride)
{
    int64_t x;
    if (given < 0) return WKV7_ERR_INVALID;
    *stride = given ? given : heads * D;
    if (*stride < heads * D || *stride % 8 != 0) return WKV7_ERR_INVALID;
    if (*stride > kMaxStride) return WKV7_ERR_UNSUPPORTED;
    if (!mul_ok(tokens, *stride * 4, &x)) return WKV7_ERR_INVALID;
    return WKV7_OK;
}

int check_heads(int64_t Hq, int64_t Hk, int64_t D)
{
    if (Hq < 0 || Hk < 0 || D <= 0) return WKV7_ERR_INVALID;
    if (Hk == 0 ? Hq != 0 : Hq == 0 || Hq % Hk != 0) return WKV7_ERR_INVALID;
    if ((D != 64 && D != 128) || Hq > 65535) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

int check(const attn_shape *s, wkv7::attn::Launch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->B < 0 || s->T < 0 || s->nseq < 0 || s->flags != 0 || !is_dtype(s->dtype)) return WKV7_ERR_INVALID;
    if (!is_scale(s->scale)) return WKV7_ERR_INVALID;
    if (s->nseq > 0 && s->B != 1) return WKV7_ERR_INVALID;
    int rc = check_heads(s->Hq, s->Hk, s->D);
    if (rc != WKV7_OK) return rc;
    if (s->T > kMaxTokens || s->nseq > 65535) return WKV7_ERR_UNSUPPORTED;
    int64_t tokens, x;
    if (!mul_ok(s->B, s->T, &tokens)) return WKV7_ERR_INVALID;
    if ((rc = check_stride(s->q_stride, s->Hq, s->D, tokens, &L->q_stride)) != WKV7_OK) return rc;
    if ((rc = check_stride(s->k_stride, s->Hk, s->D, tokens, &L->k_stride)) != WKV7_OK) return rc;
    if ((rc = check_stride(s->v_stride, s->Hk, s->D, tokens, &L->v_stride)) != WKV7_OK) return rc;
    const int64_t tiles = (s->T + wkv7::attn::kTile - 1) / wkv7::attn::kTile;
    int64_t slots = s->T / wkv7::attn::kTile + s->nseq;
    if (s->nseq == 0 && !mul_ok(s->B, tiles, &slots)) return WKV7_ERR_INVALID;
    if (!mul_ok(slots, s->Hq, &x)) return WKV7_ERR_INVALID;
    if (x > kMaxBlocks) return WKV7_ERR_UNSUPPORTED;
    L->seqs = {nullptr, s->T, s->nseq > 0 ? s->nseq : s->B, tiles, slots};
    L->B = s->B;
    L->Hq = s->Hq;
    L->Hk = s->Hk;
    L->D = s->D;
    L->dtype = s->dtype;
    L->scale = s->scale;
    return WKV7_OK;
}

bool has_tokens(const wkv7::attn::Launch &L) { return L.B > 0 && L.seqs.T > 0 && L.Hq > 0; }
size_t entries(const wkv7::attn::Launch &L) { return (size_t)(L.B * L.seqs.T * L.Hq); }
size_t stats_bytes(const wkv7::attn::Launch &L) { return round_up(entries(L) * 8); }

int set_starts(const attn_shape *s, const int32_t *starts, wkv7::attn::Launch *L)
{
    if ((s->nseq > 0) != (starts != nullptr) || !aligned(starts, 4)) return WKV7_ERR_INVALID;
    L->seqs.starts = starts;
    return WKV7_OK;
}

int check(const qk_norm_shape *s, wkv7::attn::QkNormLaunch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->B < 0 || s->T < 0 || s->Hq < 0 || s->Hk < 0 || s->D <= 0 || s->R < 0 || !is_dtype(s->dtype))
        return WKV7_ERR_INVALID;
    if ((s->flags & ~QK_NORM_INTERLEAVED) != 0 || !(s->eps > 0.f) || !std::isfinite(s->eps)) return WKV7_ERR_INVALID;
    if ((s->D != 64 && s->D != 128) || s->Hq > 65535 || s->Hk > 65535) return WKV7_ERR_UNSUPPORTED;
    if (s->R > s->D) return WKV7_ERR_INVALID;
    if (s->R % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    int64_t tokens;
    int rc;
    if (!mul_ok(s->B, s->T, &tokens)) return WKV7_ERR_INVALID;
    if ((rc = check_stride(s->q_stride, s->Hq, s->D, tokens, &L->q_stride)) != WKV7_OK) return rc;
    if ((rc = check_stride(s->k_stride, s->Hk, s->D, tokens, &L->k_stride)) != WKV7_OK) return rc;
    L->B = s->B;
    L->T = s->T;
    L->Hq = s->Hq;
    L->Hk = s->Hk;
    L->D = s->D;
    L->R = s->R;
    L->dtype = s->dtype;
    L->interleaved = (s->flags & QK_NORM_INTERLEAVED) != 0;
    L->eps = s->eps;
    return WKV7_OK;
}

size_t part_bytes(const wkv7::attn::QkNormLaunch &L)
{
    return round_up((size_t)wkv7::attn::qk_norm_parts(L.B * L.T) * 2 * (size_t)L.D * 4);
}

// Weights come together, the angles' rates with entries that turn.
int check_qk(const wkv7::attn::QkNormLaunch &L, const float *wq, const float *wk, const float *theta,
             const int32_t *positions)
{
    if ((wq != nullptr) != (wk != nullptr) || !aligned(wq) || !aligned(wk)) return WKV7_ERR_INVALID;
    if ((theta != nullptr) != (L.R > 0) || !aligned(theta, 4) || !aligned(positions, 4)) return WKV7_ERR_INVALID;
    return WKV7_OK;
}

struct Pool {
    int64_t pages, page, max_pages, Hk, D, rows;
    int32_t cache_dtype;
};

int check_pool(const Pool &p)
{
    int64_t x;
    if (p.pages < 0 || p.page <= 0 || p.max_pages < 0 || p.rows < 0 || !is_cache(p.cache_dtype)) return WKV7_ERR_INVALID;
    if (p.pages > INT32_MAX || p.page < 16 || p.page > 256 || (p.page & (p.page - 1)) != 0) return WKV7_ERR_UNSUPPORTED;
    if (!mul_ok(p.max_pages, p.page, &x)) return WKV7_ERR_INVALID;
    if (x > kMaxTokens) return WKV7_ERR_UNSUPPORTED;
    if (!mul_ok(p.pages, p.page * (p.Hk + 1) * p.D * 4, &x) || !mul_ok(p.rows, (p.max_pages + 1) * 4, &x))
        return WKV7_ERR_INVALID;
    return WKV7_OK;
}

int check_scales(int32_t cache_dtype, const float *k_scale, const float *v_scale)
{
    const bool need = cache_dtype == KV_CACHE_E4M3;
    if ((k_scale != nullptr) != need || (v_scale != nullptr) != need) return WKV7_ERR_INVALID;
    return aligned(k_scale, 4) && aligned(v_scale, 4) ? WKV7_OK : WKV7_ERR_INVALID;
}

int check(const kv_cache_shape *s, wkv7::attn::CacheLaunch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->T < 0 || s->Hk < 0 || s->D <= 0 || (s->packed != 0 && s->packed != 1) || !is_dtype(s->dtype))
        return WKV7_ERR_INVALID;
    if ((s->D != 64 && s->D != 128) || s->Hk > 65535) return WKV7_ERR_UNSUPPORTED;
    int rc = check_pool({s->pages, s->page, s->max_pages, s->Hk, s->D, s->rows, s->cache_dtype});
    if (rc != WKV7_OK) return rc;
    if (s->rows > INT32_MAX || s->T > INT32_MAX) return WKV7_ERR_UNSUPPORTED;
    L->tokens = s->packed ? s->T : s->rows * s->T;
    if (L->tokens > INT32_MAX) return WKV7_ERR_UNSUPPORTED;
    if ((rc = check_stride(s->k_stride, s->Hk, s->D, L->tokens, &L->k_stride)) != WKV7_OK) return rc;
    if ((rc = check_stride(s->v_stride, s->Hk, s->D, L->tokens, &L->v_stride)) != WKV7_OK) return rc;
    L->rows = s->rows;
    L->T = s->T;
    L->Hk = s->Hk;
    L->D = s->D;
    L->pages = s->pages;
    L->page = s->page;
    L->max_pages = s->max_pages;
    L->dtype = s->dtype;
    L->cache_dtype = s->cache_dtype;
    return WKV7_OK;
}

// Whether there is anything to do; tokens that nobody owns are nothing.
bool has_tokens(const wkv7::attn::CacheLaunch &L) { return L.rows > 0 && L.tokens > 0 && L.Hk > 0; }

int set_cache(const kv_cache_shape *s, const void *k, const void *v, const void *k_pages, const void *v_pages,
              const float *k_scale, const float *v_scale, const int32_t *table, const int32_t *lens,
              const int32_t *starts, wkv7::attn::CacheLaunch *L)
{
    for (const void *p : {k, v, k_pages, v_pages})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    for (const int32_t *p : {table, lens, starts})
        if (!aligned(p, 4)) return WKV7_ERR_INVALID;
    if (s->packed ? L->rows > 0 && !starts : starts != nullptr) return WKV7_ERR_INVALID;
    if (!has_tokens(*L)) return WKV7_OK;
    if (!k || !v || !lens || (L->max_pages > 0 && !table)) return WKV7_ERR_INVALID;
    if (L->pages > 0) {
        if (!k_pages || !v_pages) return WKV7_ERR_INVALID;
        const int rc = check_scales(s->cache_dtype, k_scale, v_scale);
        if (rc != WKV7_OK) return rc;
    }
    L->k = k;
    L->v = v;
    L->k_pages = k_pages;
    L->v_pages = v_pages;
    L->k_scale = const_cast<float *>(k_scale);
    L->v_scale = const_cast<float *>(v_scale);
    L->table = table;
    L->lens = lens;
    L->starts = starts;
    return WKV7_OK;
}

int check(const attn_decode_shape *s, wkv7::attn::DecodeLaunch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->B < 0 || s->T < 0 || !is_dtype(s->dtype)) return WKV7_ERR_INVALID;
    if (!is_scale(s->scale)) return WKV7_ERR_INVALID;
    int rc = check_heads(s->Hq, s->Hk, s->D);
    if (rc != WKV7_OK) return rc;
    rc = check_pool({s->pages, s->page, s->max_pages, s->Hk, s->D, s->B, s->cache_dtype});
    if (rc != WKV7_OK) return rc;
    if (s->B > 65535 || s->T > 65535) return WKV7_ERR_UNSUPPORTED;
    if ((rc = check_stride(s->q_stride, s->Hq, s->D, s->B * s->T, &L->q_stride)) != WKV7_OK) return rc;
    L->B = s->B;
    L->T = s->T;
    L->Hq = s->Hq;
    L->Hk = s->Hk;
    L->D = s->D;
    L->pages = s->pages;
    L->page = s->page;
    L->max_pages = s->max_pages;
    L->dtype = s->dtype;
    L->cache_dtype = s->cache_dtype;
    L->scale = s->scale;
    L->splits = 1;
    if (s->B == 0 || s->T == 0 || s->Hq == 0) return WKV7_OK;
    const int64_t rows = s->T * (s->Hq / s->Hk);
    if ((rows + wkv7::attn::kDecodeRows - 1) / wkv7::attn::kDecodeRows * s->Hk > 65535) return WKV7_ERR_UNSUPPORTED;
    L->splits = wkv7::attn::decode_splits(s->B, s->T, s->Hq, s->Hk, s->max_pages * s->page);
    return WKV7_OK;
}

bool has_tokens(const wkv7::attn::DecodeLaunch &L) { return L.B > 0 && L.T > 0 && L.Hq > 0; }
size_t parts(const wkv7::attn::DecodeLaunch &L)
{
    return has_tokens(L) && L.splits > 1 ? (size_t)(L.B * L.T * L.Hq * L.splits) : 0;
}
size_t decode_bytes(const wkv7::attn::DecodeLaunch &L)
{
    return round_up(parts(L) * (size_t)L.D * 4) + round_up(parts(L) * 8);
}

}  // namespace

extern "C" {

size_t attn_record_bytes(const attn_shape *shape)
{
    wkv7::attn::Launch L;
    if (check(shape, &L) != WKV7_OK || !has_tokens(L) || L.dtype != WKV7_BF16) return 0;
    return entries(L) * (size_t)L.D * 2;
}

size_t attn_backward_workspace_bytes(const attn_shape *shape)
{
    wkv7::attn::Launch L;
    if (check(shape, &L) != WKV7_OK || !has_tokens(L)) return 0;
    return stats_bytes(L);
}

int attn_forward(const attn_shape *shape, const void *q, const void *k, const void *v,
                 const int32_t *seq_starts, void *y, float *lse, void *record, hipStream_t stream)
{
    wkv7::attn::Launch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK) rc = set_starts(shape, seq_starts, &L);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {q, k, v, (const void *)y, (const void *)record})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (!aligned(lse, 4) || (record && L.dtype != WKV7_BF16)) return WKV7_ERR_INVALID;
    if (!has_tokens(L)) return WKV7_OK;
    if (!q || !k || !v || !y) return WKV7_ERR_INVALID;
    L.q = q;
    L.k = k;
    L.v = v;
    L.y = y;
    L.lse = lse;
    L.record = record;
    return status(wkv7::attn::launch_forward(L, stream));
}

int attn_backward(const attn_shape *shape, const void *q, const void *k, const void *v,
                  const int32_t *seq_starts, const void *y, const float *lse, const void *record,
                  const void *dy, void *dq, void *dk, void *dv, void *workspace,
                  size_t workspace_bytes, hipStream_t stream)
{
    wkv7::attn::Launch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK) rc = set_starts(shape, seq_starts, &L);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {q, k, v, y, record, dy, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (!aligned(lse, 4) || (record && L.dtype != WKV7_BF16)) return WKV7_ERR_INVALID;
    if (!has_tokens(L)) return WKV7_OK;
    for (const void *p : {q, k, v, y, (const void *)lse, dy, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!p) return WKV7_ERR_INVALID;
    rc = check_workspace(workspace, workspace_bytes, stats_bytes(L));
    if (rc != WKV7_OK) return rc;
    L.q = q;
    L.k = k;
    L.v = v;
    L.y = const_cast<void *>(y);
    L.lse = const_cast<float *>(lse);
    L.record = const_cast<void *>(record);
    L.dy = dy;
    L.dq = dq;
    L.dk = dk;
    L.dv = dv;
    L.stats = static_cast<float *>(workspace);
    return status(wkv7::attn::launch_backward(L, stream));
}

size_t qk_norm_workspace_bytes(const qk_norm_shape *shape)
{
    wkv7::attn::QkNormLaunch L;
    if (check(shape, &L) != WKV7_OK || L.B * L.T == 0) return 0;
    return part_bytes(L);
}

int qk_norm_forward(const qk_norm_shape *shape, const void *q, const void *k, const float *wq,
                    const float *wk, const float *theta, const int32_t *positions, void *qz,
                    void *kz, hipStream_t stream)
{
    wkv7::attn::QkNormLaunch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK) rc = check_qk(L, wq, wk, theta, positions);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {q, k, (const void *)qz, (const void *)kz})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (L.B * L.T == 0 || L.Hq + L.Hk == 0) return WKV7_OK;
    if ((L.Hq > 0 && (!q || !qz)) || (L.Hk > 0 && (!k || !kz))) return WKV7_ERR_INVALID;
    L.q = q;
    L.k = k;
    L.wq = wq;
    L.wk = wk;
    L.theta = theta;
    L.positions = positions;
    L.qz = qz;
    L.kz = kz;
    return status(wkv7::attn::launch_qk_norm_forward(L, stream));
}

int qk_norm_backward(const qk_norm_shape *shape, const void *dqz, const void *dkz, const void *q,
                     const void *k, const float *wq, const float *wk, const float *theta,
                     const int32_t *positions, void *dq, void *dk, float *dwq, float *dwk,
                     void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    wkv7::attn::QkNormLaunch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK) rc = check_qk(L, wq, wk, theta, positions);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {dqz, dkz, q, k, (const void *)dq, (const void *)dk, (const void *)dwq, (const void *)dwk})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if ((wq != nullptr) != (dwq != nullptr) || (wk != nullptr) != (dwk != nullptr)) return WKV7_ERR_INVALID;
    if (L.B * L.T == 0) {
        if (!dwq) return WKV7_OK;
        rc = status(wkv7::launch_fill(dwq, nullptr, (size_t)L.D, stream));
        return rc == WKV7_OK ? status(wkv7::launch_fill(dwk, nullptr, (size_t)L.D, stream)) : rc;
    }
    if (L.Hq > 0 && (!dqz || !dq || !q)) return WKV7_ERR_INVALID;
    if (L.Hk > 0 && (!dkz || !dk || !k)) return WKV7_ERR_INVALID;
    rc = check_workspace(workspace, workspace_bytes, wq ? part_bytes(L) : 0);
    if (rc != WKV7_OK) return rc;
    L.dqz = dqz;
    L.dkz = dkz;
    L.q = q;
    L.k = k;
    L.wq = wq;
    L.wk = wk;
    L.theta = theta;
    L.positions = positions;
    L.dq = dq;
    L.dk = dk;
    L.dwq = dwq;
    L.dwk = dwk;
    L.part = static_cast<float *>(workspace);
    return status(wkv7::attn::launch_qk_norm_backward(L, stream));
}

int kv_write(const kv_cache_shape *shape, const void *k, const void *v, void *k_pages,
             void *v_pages, float *k_scale, float *v_scale, const int32_t *table,
             const int32_t *lens, const int32_t *seq_starts, hipStream_t stream)
{
    wkv7::attn::CacheLaunch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK) rc = set_cache(shape, k, v, k_pages, v_pages, k_scale, v_scale, table, lens, seq_starts, &L);
    if (rc != WKV7_OK || !has_tokens(L) || L.pages == 0 || L.max_pages == 0) return rc;
    L.k_out = k_pages;
    L.v_out = v_pages;
    return status(wkv7::attn::launch_kv_write(L, stream));
}

int kv_read(const kv_cache_shape *shape, const void *k_pages, const void *v_pages,
            const float *k_scale, const float *v_scale, const int32_t *table,
            const int32_t *lens, const int32_t *seq_starts, void *k, void *v, hipStream_t stream)
{
    wkv7::attn::CacheLaunch L;
    int rc = check(shape, &L);
    if (rc == WKV7_OK && (shape->k_stride || shape->v_stride)) rc = WKV7_ERR_INVALID;
    if (rc == WKV7_OK) rc = set_cache(shape, k, v, k_pages, v_pages, k_scale, v_scale, table, lens, seq_starts, &L);
    if (rc != WKV7_OK || !has_tokens(L)) return rc;
    L.k_out = k;
    L.v_out = v;
    return status(wkv7::attn::launch_kv_read(L, stream));
}

size_t attn_decode_workspace_bytes(const attn_decode_shape *shape)
{
    wkv7::attn::DecodeLaunch L;
    return check(shape, &L) == WKV7_OK ? decode_bytes(L) : 0;
}

int attn_decode(const attn_decode_shape *shape, const void *q, const void *k_pages,
                const void *v_pages, const float *k_scale, const float *v_scale,
                const int32_t *table, const int32_t *lens, void *y, void *workspace,
                size_t workspace_bytes, hipStream_t stream)
{
    wkv7::attn::DecodeLaunch L;
    int rc = check(shape, &L);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {q, k_pages, v_pages, (const void *)y})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (!aligned(table, 4) || !aligned(lens, 4)) return WKV7_ERR_INVALID;
    if (!has_tokens(L)) return WKV7_OK;
    if (!q || !y || !lens || (L.max_pages > 0 && !table)) return WKV7_ERR_INVALID;
    if (L.pages > 0) {
        if (!k_pages || !v_pages) return WKV7_ERR_INVALID;
        rc = check_scales(L.cache_dtype, k_scale, v_scale);
        if (rc != WKV7_OK) return rc;
    }
    rc = check_workspace(workspace, workspace_bytes, decode_bytes(L));
    if (rc != WKV7_OK) return rc;
    L.q = q;
    L.k_pages = k_pages;
    L.v_pages = v_pages;
    L.k_scale = k_scale;
    L.v_scale = v_scale;
    L.table = table;
    L.lens = lens;
    L.y = y;
    char *ws = static_cast<char *>(workspace);
    L.part_o = parts(L) ? reinterpret_cast<float *>(ws) : nullptr;
    L.part_ml = parts(L) ? reinterpret_cast<float *>(ws + round_up(parts(L) * (size_t)L.D * 4)) : nullptr;
    return status(wkv7::attn::launch_decode(L, stream));
}

}  // extern "C"
