// Host-only driver for the validation and the buffer layout of the gated
// delta rule, its epilogue and the residual norm, built with AddressSanitizer
// and UndefinedBehaviorSanitizer (tests/test_sanitize_gdr_cpu.py).  The kernel
// launchers are replaced by stubs that record what they were given; the
// driver checks that every part of a record or workspace that a kernel is
// handed lies inside the sizes the ABI reports, and apart from the others.
// No GPU is used.
#include <cstdio>
#include <utility>
#include <vector>

#include "gdr_internal.h"
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

using wkv7::gdr::Launch;
std::vector<Launch> g_scan, g_reverse, g_grads;
std::vector<wkv7::gdr::EpilogueLaunch> g_epi;
std::vector<wkv7::gdr::NormLaunch> g_norm;
constexpr size_t kFactor = 26 * 1024, kFactorT = 31 * 1024;
}  // namespace

namespace wkv7 {
hipError_t launch_fill(float *, const float *, size_t, hipStream_t) { return hipSuccess; }
namespace gdr {
size_t factor_bytes(int, bool transposed) { return transposed ? kFactorT : kFactor; }
hipError_t launch_scan(const Launch &a, hipStream_t) { g_scan.push_back(a); return hipSuccess; }
hipError_t launch_reverse(const Launch &a, hipStream_t) { g_reverse.push_back(a); return hipSuccess; }
hipError_t launch_grads(const Launch &a, hipStream_t) { g_grads.push_back(a); return hipSuccess; }
hipError_t launch_decode(const DecodeLaunch &, hipStream_t) { return hipSuccess; }
int64_t epilogue_parts(int64_t, int64_t, int64_t, int64_t) { return 7; }
hipError_t launch_epilogue_forward(const EpilogueLaunch &, hipStream_t) { return hipSuccess; }
hipError_t launch_epilogue_backward(const EpilogueLaunch &a, hipStream_t) { g_epi.push_back(a); return hipSuccess; }
int64_t norm_parts(int64_t, int64_t) { return 5; }
hipError_t launch_norm_forward(const NormLaunch &, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_backward(const NormLaunch &a, hipStream_t) { g_norm.push_back(a); return hipSuccess; }
}  // namespace gdr
}  // namespace wkv7

namespace {
char *const kWs = reinterpret_cast<char *>(uintptr_t(1) << 40);
float *const kRec = reinterpret_cast<float *>(uintptr_t(1) << 44);
float *const kIn = reinterpret_cast<float *>(uintptr_t(1) << 20);

using Span = std::pair<const void *, size_t>;
// The spans that are there lie in [base, base + size) and apart.
void check_spans(const std::vector<Span> &spans, const void *base, size_t size)
{
    const uintptr_t lo = (uintptr_t)base, hi = lo + size;
    for (size_t i = 0; i < spans.size(); ++i) {
        if (!spans[i].first || !spans[i].second) continue;
        const uintptr_t a = (uintptr_t)spans[i].first, b = a + spans[i].second;
        CHECK(a >= lo && b <= hi && a % 256 == 0);
        for (size_t j = 0; j < i; ++j) {
            if (!spans[j].first || !spans[j].second) continue;
            const uintptr_t c = (uintptr_t)spans[j].first, d = c + spans[j].second;
            CHECK(b <= c || d <= a);
        }
    }
}

void check_rule(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t K, int64_t V, int64_t nseq, int dtype)
{
    const gdr_shape s{B, T, Hk, Hv, K, V, nseq, dtype, 0, 0.125f};
    const int32_t *starts = nseq ? reinterpret_cast<const int32_t *>(kIn) : nullptr;
    const size_t rec = gdr_checkpoint_bytes(&s), fw = gdr_forward_workspace_bytes(&s);
    g_scan.clear();
    CHECK(gdr_forward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, kIn, kRec, kWs, fw, nullptr) == WKV7_OK);
    if (fw) CHECK(gdr_forward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, kIn, kRec, kWs, fw - 1, nullptr) ==
                  WKV7_ERR_WORKSPACE);
    CHECK(g_scan.size() == 1);
    const Launch &f = g_scan[0];
    const size_t per = (size_t)(f.map.slots * Hv), states = per * K * V * 4, rows = per * 64 * V * 4;
    const size_t segs = (size_t)(f.map.nseq * f.map.nseg * Hv), map = segs * K * (V + K) * 4, carry = segs * K * V * 4;
    CHECK(f.map.slots >= (nseq ? T / 64 + nseq : B * ((T + 63) / 64)));
    CHECK(f.map.nseg >= 1 && f.map.nckseg * f.map.nseg >= f.map.nck && f.map.nckseg * (f.map.nseg - 1) < f.map.nck);
    if (f.map.nseg > 1) CHECK(f.factors && f.seg_map && f.carry && !nseq);
    check_spans({{f.rec_s, states}, {f.rec_e, rows}}, kRec, rec);
    check_spans({{f.factors, per * kFactor}, {f.seg_map, map}, {f.carry, carry}}, kWs, fw);
    for (int given = 0; given < 2; ++given) {
        const size_t bw = gdr_backward_workspace_bytes(&s, given);
        g_scan.clear();
        g_reverse.clear();
        g_grads.clear();
        float *const ck = given ? kRec : nullptr;
        CHECK(gdr_backward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, nullptr, ck, kIn, kIn, kIn, kIn, kIn,
                           nullptr, kWs, bw, nullptr) == WKV7_OK);
        CHECK(gdr_backward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, nullptr, ck, kIn, kIn, kIn, kIn, kIn,
                           nullptr, kWs, bw - 1, nullptr) == WKV7_ERR_WORKSPACE);
        CHECK(g_scan.size() == (given ? 0u : 1u) && g_reverse.size() == 1 && g_grads.size() == 1);
        const Launch &r = g_reverse[0];
        const std::vector<Span> own = {{r.table, per * 5 * 64 * 4}, {r.factors, per * kFactorT}, {r.seg_map, map},
                                       {r.carry, carry}, {r.ws_ds, states}, {r.ws_dr, rows}};
        std::vector<Span> all = own;
        if (given)
            check_spans({{r.rec_s, states}, {r.rec_e, rows}}, kRec, rec);
        else
            all.insert(all.end(), {{r.rec_s, states}, {r.rec_e, rows}});
        check_spans(all, kWs, bw);
    }
}
}  // namespace

int main()
{
    for (int dtype : {WKV7_F32, WKV7_BF16})
        for (int64_t K : {64, 128})
            for (int64_t V : {16, 48, 64, 128, 256})
                for (int64_t Hv : {1, 6, 128})
                    for (int64_t T : {1, 63, 64, 65, 1000, 4096, 70000}) {
                        check_rule(1, T, 1, Hv, K, V, 0, dtype);
                        check_rule(3, T, Hv, Hv, K, V, 0, dtype);
                        check_rule(1, T, 1, Hv, K, V, 1, dtype);
                        check_rule(1, T, Hv, Hv, K, V, 50, dtype);
                    }
    // sizes whose products pass 64 bits are refused, not wrapped
    const int64_t big = INT64_MAX;
    for (int64_t B : {int64_t(1), int64_t(65535), big / 2, big})
        for (int64_t T : {int64_t(1), int64_t(1) << 40, big / 3, big})
            for (int64_t H : {int64_t(1), int64_t(65535), big}) {
                const gdr_shape s{B, T, H, H, 128, 256, 0, WKV7_BF16, 0, 1.f};
                gdr_checkpoint_bytes(&s);
                gdr_backward_workspace_bytes(&s, 0);
                CHECK(gdr_decode(&s, kIn, kIn, kIn, kIn, kIn, kIn, big, nullptr, kIn, nullptr) != WKV7_OK);
                const gdr_epilogue_shape e{B, T, 64, 1, WKV7_BF16, 0, 1e-6f};
                gdr_epilogue_workspace_bytes(&e);
                const residual_norm_shape n{T, 16384, WKV7_BF16, 0, 1e-6f};
                residual_norm_workspace_bytes(&n);
            }
    const gdr_epilogue_shape e{1000, 8, 64, 8, WKV7_BF16, 0, 1e-6f};
    size_t n = gdr_epilogue_workspace_bytes(&e);
    CHECK(gdr_epilogue_backward(&e, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, n, nullptr) == WKV7_OK && g_epi.size() == 1);
    check_spans({{g_epi[0].part, (size_t)(8 * 7 * 64 * 4)}}, kWs, n);
    const residual_norm_shape r{1000, 2047, WKV7_F32, 0, 1e-6f};
    n = residual_norm_workspace_bytes(&r);
    CHECK(residual_norm_backward(&r, kIn, nullptr, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, n, nullptr) == WKV7_OK &&
          g_norm.size() == 1);
    check_spans({{g_norm[0].part, (size_t)(5 * 2 * 2047 * 4)}}, kWs, n);
    return g_fails ? 1 : 0;
}
