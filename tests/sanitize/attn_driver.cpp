// Host-only driver for the validation and the workspace layout of softmax
// attention, the norm before it and the paged cache, built with
// AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_sanitize_attn_cpu.py).  The kernel launchers are replaced by stubs
// that record what they were given; the driver checks that every part of a
// workspace that a kernel is handed lies inside the size the ABI reports, apart
// from the others, and that launches fit the grids and index widths the kernels
// assume, over ordinary and extreme shapes.  No GPU is used.
#include <cstdio>
#include <limits>
#include <utility>
#include <vector>

#include "attn_internal.h"
#include "wkv7_internal.h"

namespace {
int g_fails = 0;
#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            std::fprintf(stderr, "CHECK failed line %d: %s\n", __LINE__, #c); \
            ++g_fails;                                                        \
        }                                                                     \
    } while (0)

using namespace wkv7::attn;
std::vector<Launch> g_fwd, g_bwd;
std::vector<QkNormLaunch> g_norm;
std::vector<CacheLaunch> g_cache;
std::vector<DecodeLaunch> g_decode;
int g_fills = 0;
}  // namespace

namespace wkv7 {
hipError_t launch_fill(float *, const float *, size_t, hipStream_t)
{
    ++g_fills;
    return hipSuccess;
}
namespace attn {
hipError_t launch_forward(const Launch &a, hipStream_t) { g_fwd.push_back(a); return hipSuccess; }
hipError_t launch_backward(const Launch &a, hipStream_t) { g_bwd.push_back(a); return hipSuccess; }
hipError_t launch_qk_norm_forward(const QkNormLaunch &a, hipStream_t) { g_norm.push_back(a); return hipSuccess; }
hipError_t launch_qk_norm_backward(const QkNormLaunch &a, hipStream_t) { g_norm.push_back(a); return hipSuccess; }
hipError_t launch_kv_write(const CacheLaunch &a, hipStream_t) { g_cache.push_back(a); return hipSuccess; }
hipError_t launch_kv_read(const CacheLaunch &a, hipStream_t) { g_cache.push_back(a); return hipSuccess; }
hipError_t launch_decode(const DecodeLaunch &a, hipStream_t) { g_decode.push_back(a); return hipSuccess; }
}  // namespace attn
}  // namespace wkv7

namespace {
char *const kWs = reinterpret_cast<char *>(uintptr_t(1) << 40);
float *const kIn = reinterpret_cast<float *>(uintptr_t(1) << 20);
int32_t *const kInt = reinterpret_cast<int32_t *>(uintptr_t(1) << 20);
constexpr int64_t kHuge = std::numeric_limits<int64_t>::max();

using Span = std::pair<const void *, size_t>;
// The spans that are there lie in [kWs, kWs + size) and apart.
void check_spans(const std::vector<Span> &spans, size_t size)
{
    const uintptr_t lo = (uintptr_t)kWs, hi = lo + size;
    for (size_t i = 0; i < spans.size(); ++i) {
        const uintptr_t a = (uintptr_t)spans[i].first, b = a + spans[i].second;
        CHECK(a >= lo && b <= hi && a % 256 == 0);
        for (size_t j = 0; j < i; ++j) {
            const uintptr_t c = (uintptr_t)spans[j].first, d = c + spans[j].second;
            CHECK(b <= c || d <= a);
        }
    }
}

void check_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t nseq, int64_t stride, int dtype)
{
    const attn_shape s{B, T, Hq, Hk, D, nseq, stride, stride, 0, dtype, 0, 0.125f};
    const int32_t *starts = nseq ? kInt : nullptr;
    void *const rec = dtype == WKV7_BF16 ? kIn : nullptr;
    const size_t ws = attn_backward_workspace_bytes(&s);
    g_fwd.clear();
    g_bwd.clear();
    const int rc = attn_forward(&s, kIn, kIn, kIn, starts, kIn, kIn, rec, nullptr);
    CHECK(attn_backward(&s, kIn, kIn, kIn, starts, kIn, kIn, rec, kIn, kIn, kIn, kIn, kWs, ws, nullptr) == rc);
    if (rc != WKV7_OK) {
        CHECK(g_fwd.empty() && g_bwd.empty() && ws == 0 && attn_record_bytes(&s) == 0);
        return;
    }
    if (B * T * Hq == 0) {
        CHECK(g_fwd.empty() && g_bwd.empty() && ws == 0);
        return;
    }
    CHECK(g_fwd.size() == 1 && g_bwd.size() == 1);
    CHECK(attn_backward(&s, kIn, kIn, kIn, starts, kIn, kIn, rec, kIn, kIn, kIn, kIn, kWs, ws - 1, nullptr) ==
          WKV7_ERR_WORKSPACE);
    CHECK(attn_record_bytes(&s) == (rec ? (size_t)(B * T * Hq * D) * 2 : 0));
    const Launch &a = g_bwd[0];
    check_spans({{a.stats, (size_t)(Hq * B * T) * 8}}, ws);
    // grids, also of the narrow form, and the indexes the kernels keep in 32 bits
    const int64_t narrow = nseq ? T / 32 + nseq : B * ((T + 31) / 32), tiles = (T + kTile - 1) / kTile;
    CHECK(a.seqs.slots >= (nseq ? T / kTile + nseq : B * tiles) && a.seqs.tiles == tiles);
    CHECK(a.seqs.slots * Hq < (int64_t(1) << 24) && narrow * Hq < (int64_t(1) << 32) / 256 * 5);
    if (is_narrow(a.seqs.slots * Hq, dtype)) CHECK(narrow * Hq < 512 * 5);
    CHECK(T + 256 < std::numeric_limits<int32_t>::max());
    for (int64_t stride_ : {a.q_stride, a.k_stride, a.v_stride, Hq * D})
        CHECK(stride_ * 4 * 64 < (int64_t(1) << 32) && stride_ % 8 == 0);
}

void check_norm(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int dtype)
{
    const qk_norm_shape s{B, T, Hq, Hk, D, R, 0, 0, dtype, QK_NORM_INTERLEAVED, 1e-6f};
    const float *theta = R ? kIn : nullptr;
    const size_t ws = qk_norm_workspace_bytes(&s);
    g_norm.clear();
    g_fills = 0;
    const int rc = qk_norm_forward(&s, kIn, kIn, kIn, kIn, theta, nullptr, kIn, kIn, nullptr);
    CHECK(qk_norm_backward(&s, kIn, kIn, kIn, kIn, kIn, kIn, theta, kInt, kIn, kIn, kIn, kIn, kWs, ws, nullptr) == rc);
    if (rc != WKV7_OK) {
        CHECK(g_norm.empty() && ws == 0);
        return;
    }
    if (B * T == 0) {   // the weights' gradients are zeros
        CHECK(g_norm.empty() && ws == 0 && g_fills == 2);
        return;
    }
    CHECK(g_norm.size() == (Hq + Hk ? 2u : 1u));
    CHECK(qk_norm_backward(&s, kIn, kIn, kIn, kIn, kIn, kIn, theta, kInt, kIn, kIn, kIn, kIn, kWs, ws - 1, nullptr) ==
          WKV7_ERR_WORKSPACE);
    CHECK(qk_norm_backward(&s, kIn, kIn, kIn, kIn, nullptr, nullptr, theta, kInt, kIn, kIn, nullptr, nullptr, nullptr, 0,
                           nullptr) == WKV7_OK);
    check_spans({{kWs, (size_t)qk_norm_parts(B * T) * 2 * D * 4}}, ws);
    CHECK(g_norm[0].q_stride == Hq * D);
}

void check_decode(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t pages, int64_t page,
                  int64_t max_pages, int dtype, int kind)
{
    const attn_decode_shape s{B, T, Hq, Hk, D, pages, page, max_pages, 0, dtype, kind, 0.125f};
    const float *scale = kind == KV_CACHE_E4M3 ? kIn : nullptr;
    const size_t ws = attn_decode_workspace_bytes(&s);
    g_decode.clear();
    const int rc = attn_decode(&s, kIn, kIn, kIn, scale, scale, kInt, kInt, kIn, kWs, ws, nullptr);
    if (rc != WKV7_OK || B * T * Hq == 0) {
        CHECK(g_decode.empty() && ws == 0);
        return;
    }
    CHECK(g_decode.size() == 1);
    const DecodeLaunch &a = g_decode[0];
    const size_t parts = (size_t)(B * T * Hq * a.splits);
    CHECK((a.splits > 1) == (a.part_o != nullptr) && (ws != 0) == (a.splits > 1));
    if (a.splits > 1) {
        check_spans({{a.part_o, parts * D * 4}, {a.part_ml, parts * 8}}, ws);
        CHECK(attn_decode(&s, kIn, kIn, kIn, scale, scale, kInt, kInt, kIn, kWs, ws - 1, nullptr) == WKV7_ERR_WORKSPACE);
        CHECK(attn_decode(&s, kIn, kIn, kIn, scale, scale, kInt, kInt, kIn, kWs + 16, ws, nullptr) == WKV7_ERR_WORKSPACE);
    }
    const int64_t rows = T * (Hq / Hk), tiles = (rows + kDecodeRows - 1) / kDecodeRows;
    CHECK(B <= 65535 && Hk * tiles <= 65535 && a.splits >= 1 && a.splits <= 512);
    CHECK(max_pages * page <= (int64_t(1) << 30));
}

void check_cache(int64_t rows, int64_t T, int64_t Hk, int64_t D, int64_t packed, int64_t pages, int64_t page,
                 int64_t max_pages, int dtype, int kind)
{
    const kv_cache_shape s{rows, T, Hk, D, packed, pages, page, max_pages, 0, 0, dtype, kind};
    float *scale = kind == KV_CACHE_E4M3 ? kIn : nullptr;
    const int32_t *starts = packed ? kInt : nullptr;
    g_cache.clear();
    const int rc = kv_write(&s, kIn, kIn, kIn, kIn, scale, scale, kInt, kInt, starts, nullptr);
    CHECK(kv_read(&s, kIn, kIn, scale, scale, kInt, kInt, starts, kIn, kIn, nullptr) == rc);
    if (rc != WKV7_OK) {
        CHECK(g_cache.empty());
        return;
    }
    for (const CacheLaunch &a : g_cache) {
        CHECK(a.tokens == (packed ? T : rows * T) && a.tokens > 0 && a.tokens <= INT32_MAX && a.Hk > 0);
        CHECK(a.rows > 0 && a.rows <= INT32_MAX && a.pages <= INT32_MAX);
        CHECK((a.page & (a.page - 1)) == 0 && a.page >= 16 && a.page <= 256);
    }
    if (rows * T * Hk == 0) CHECK(g_cache.empty());
}
}  // namespace

int main()
{
    const int64_t odd[] = {0, 1, 2, 3, 17, 65535, 65536, int64_t(1) << 30, (int64_t(1) << 30) + 1, int64_t(1) << 40, kHuge, -1};
    for (int dtype : {WKV7_F32, WKV7_BF16}) {
        for (int64_t B : {1, 2, 300})
            for (int64_t T : {1, 31, 128, 129, 4096, 70000})
                for (int64_t Hk : {1, 3, 48})
                    for (int64_t group : {1, 5})
                        for (int64_t D : {64, 128}) {
                            check_attention(B, T, Hk * group, Hk, D, 0, 0, dtype);
                            check_attention(B, T, Hk * group, Hk, D, 0, 1 << 20, dtype);
                            check_attention(1, T, Hk * group, Hk, D, B, 0, dtype);
                            check_norm(B, T, Hk * group, Hk, D, 32, dtype);
                            for (int kind : {KV_CACHE_SAME, KV_CACHE_E4M3}) {
                                check_decode(B, T < 5000 ? T : 3, Hk * group, Hk, D, 1000, 16, T, dtype, kind);
                                check_decode(B, 1, Hk * group, Hk, D, 1000, 256, 4 * T, dtype, kind);
                                check_cache(B, T, Hk, D, 0, 1000, 64, T, dtype, kind);
                                check_cache(B, T, Hk, D, 1, 1000, 64, T, dtype, kind);
                            }
                        }
        for (int64_t x : odd)
            for (int64_t y : odd) {
                check_attention(x, y, 2, 1, 64, 0, 0, dtype);
                check_attention(1, x, 4, 2, 128, y, 0, dtype);
                check_attention(1, 64, x, y, 64, 0, 0, dtype);
                check_attention(1, x, 2, 1, 64, 0, y, dtype);
                check_norm(x, y, 2, 1, 64, 0, dtype);
                check_norm(2, 2, x, y, 128, 16, dtype);
                check_norm(1, 5, 2, 2, 64, x == 3 ? 48 : x, dtype);
                check_cache(x, y, 2, 64, 0, 10, 16, 4, dtype, KV_CACHE_SAME);
                check_cache(x, y, 2, 128, 1, 10, 16, 4, dtype, KV_CACHE_E4M3);
                check_cache(2, 4, 2, 64, 0, x, 32, y, dtype, KV_CACHE_E4M3);
                check_cache(2, 4, x, 64, 0, y, 256, 4, dtype, KV_CACHE_SAME);
                check_decode(x, y, 2, 1, 64, 10, 16, 4, dtype, KV_CACHE_SAME);
                check_decode(2, 1, x, y, 128, 10, 16, 4, dtype, KV_CACHE_E4M3);
                check_decode(2, 1, 4, 2, 64, x, 64, y, dtype, KV_CACHE_SAME);
                check_decode(2, 1, 4, 2, 64, 4, x, y, dtype, KV_CACHE_E4M3);
            }
    }
    if (g_fails) std::fprintf(stderr, "%d checks failed\n", g_fails);
    return g_fails != 0;
}
