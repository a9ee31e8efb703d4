// Host-only driver for the size limits of the gated delta rule, its epilogue
// and the residual norm, built with AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_sanitize_gdr_limits_cpu.py): shapes
// beyond them are refused by every call, and their sizes are 0.  The stubs and
// CHECK are gdr_driver.cpp's.  No GPU is used.
#define main gdr_layout_main
#include "gdr_driver.cpp"
#undef main

namespace {
int64_t launches() { return (int64_t)(g_scan.size() + g_reverse.size() + g_grads.size() + g_epi.size() + g_norm.size()); }

// All calls of a shape, with everything else in order.
void refused(const gdr_shape &s)
{
    const int32_t *starts = s.nseq > 0 ? reinterpret_cast<const int32_t *>(kIn) : nullptr;
    const int64_t before = launches();
    const size_t much = SIZE_MAX;
    CHECK(gdr_checkpoint_bytes(&s) == 0);
    CHECK(gdr_forward_workspace_bytes(&s) == 0);
    CHECK(gdr_backward_workspace_bytes(&s, 0) == 0 && gdr_backward_workspace_bytes(&s, 1) == 0);
    int rc = gdr_forward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, kIn, kRec, kWs, much, nullptr);
    CHECK(rc == WKV7_ERR_INVALID || rc == WKV7_ERR_UNSUPPORTED);
    rc = gdr_backward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, starts, kIn, nullptr, kRec, kIn, kIn, kIn, kIn, kIn, nullptr,
                      kWs, much, nullptr);
    CHECK(rc == WKV7_ERR_INVALID || rc == WKV7_ERR_UNSUPPORTED);
    rc = gdr_decode(&s, kIn, kIn, kIn, kIn, kIn, kIn, 100000, reinterpret_cast<const int32_t *>(kIn), kIn, nullptr);
    CHECK(rc == WKV7_ERR_INVALID || rc == WKV7_ERR_UNSUPPORTED);
    CHECK(launches() == before);
}

// Nothing to do, whatever the other sizes: neither refused for its products
// nor launched.
void no_work(const gdr_shape &s)
{
    const int64_t before = launches();
    CHECK(gdr_checkpoint_bytes(&s) == 0 && gdr_forward_workspace_bytes(&s) == 0);
    CHECK(gdr_backward_workspace_bytes(&s, 0) == 0);
    gdr_forward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, nullptr, kIn, kIn, kRec, kWs, 1024, nullptr);
    gdr_backward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, nullptr, kIn, nullptr, kRec, kIn, kIn, kIn, kIn, kIn, nullptr,
                 kWs, 1024, nullptr);
    CHECK(launches() == before);
}

void oversized()
{
    const int64_t big = INT64_MAX;
    for (int dtype : {WKV7_F32, WKV7_BF16})
        for (int64_t V : {16, 256}) {
            for (int64_t B : {int64_t(65536), big / 2, big})
                for (int64_t T : {int64_t(1), int64_t(1) << 40, big / 3, big})
                    for (int64_t H : {int64_t(1), int64_t(65535), big}) refused({B, T, H, H, 128, V, 0, dtype, 0, 1.f});
            for (int64_t T : {int64_t(1) << 40, big / 3, big - 63, big - 62, big})
                for (int64_t H : {int64_t(1), int64_t(65535)}) {
                    refused({1, T, H, H, 64, V, 0, dtype, 0, 1.f});
                    refused({65535, T, 1, H, 64, V, 0, dtype, 0, 1.f});
                    refused({1, T, H, H, 64, V, 1, dtype, 0, 1.f});
                }
            for (int64_t n : {int64_t(65536), big / 2, big}) refused({1, 64, 1, 1, 64, V, n, dtype, 0, 1.f});
            for (int64_t T : {int64_t(0), int64_t(1), int64_t(1) << 40, big / 3, big - 63, big - 62, big}) {
                no_work({0, T, 2, 4, 64, V, 0, dtype, 0, 1.f});
                no_work({1, T, 0, 0, 64, V, 0, dtype, 0, 1.f});
            }
        }
    for (int64_t rows : {int64_t(1) << 40, big / 64, big}) {
        const gdr_epilogue_shape e{rows, 8, 64, 8, WKV7_BF16, 0, 1e-6f};
        const residual_norm_shape n{rows, 16384, WKV7_BF16, 0, 1e-6f};
        const int64_t before = launches();
        CHECK(gdr_epilogue_workspace_bytes(&e) == 0 && residual_norm_workspace_bytes(&n) == 0);
        CHECK(gdr_epilogue_forward(&e, kIn, kIn, kIn, kIn, nullptr) != WKV7_OK);
        CHECK(gdr_epilogue_backward(&e, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, SIZE_MAX, nullptr) != WKV7_OK);
        CHECK(residual_norm_forward(&n, kIn, kIn, kIn, kIn, kIn, kIn, nullptr) != WKV7_OK);
        CHECK(residual_norm_backward(&n, kIn, nullptr, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, SIZE_MAX, nullptr) !=
              WKV7_OK);
        CHECK(launches() == before);
    }
}

// At the limit of chunks times heads: what is accepted makes launches of fewer
// than 2^32 threads, and what is refused would not, or has more chunks.
void edges()
{
    const int64_t most = int64_t(1) << 32, chunks = int64_t(1) << 22;
    int accepted = 0, large = 0;
    for (int dtype : {WKV7_F32, WKV7_BF16})
        for (int64_t K : {64, 128})
            for (int64_t V = 16; V <= 256; V += 16)
                for (int64_t B : {int64_t(1), int64_t(64), int64_t(64527), int64_t(65535)})
                    for (int64_t n : {int64_t(1), int64_t(65536), chunks - 1, chunks, chunks + 1})   // chunks of a row
                        for (int64_t Hv : {int64_t(1), int64_t(56), int64_t(57), int64_t(64), int64_t(65), int64_t(65535)})
                            for (int64_t Hk : {int64_t(1), Hv})
                                for (int packed = 0; packed < 2; ++packed) {
                                    const int64_t seqs = B, rows = packed ? 1 : B;
                                    // packed: n - 1 whole chunks in all besides one for each sequence
                                    const int64_t T = packed ? 64 * (n - 1) : 64 * n - 63;
                                    if (T <= 0) continue;
                                    const gdr_shape s{rows, T, Hk, Hv, K, V, packed ? B : 0, dtype, 0, 1.f};
                                    const int64_t slots = packed ? n - 1 + B : B * n;
                                    const bool makes = wkv7::gdr::scan_makes_factors(dtype, K, V, seqs * Hv);
                                    const wkv7::gdr::ScanGrid g = wkv7::gdr::scan_grid(seqs * Hv, Hv / Hk, V, makes);
                                    const bool fits = slots * Hv <= chunks && g.blocks * g.threads < most;
                                    CHECK((gdr_checkpoint_bytes(&s) > 0) == fits);
                                    if (!fits) {
                                        const int32_t *st = packed ? reinterpret_cast<const int32_t *>(kIn) : nullptr;
                                        const size_t before = g_scan.size();
                                        const int rc = gdr_forward(&s, kIn, kIn, kIn, kIn, kIn, nullptr, st, kIn, kIn,
                                                                   kRec, kWs, SIZE_MAX, nullptr);
                                        CHECK(rc == WKV7_ERR_UNSUPPORTED || rc == WKV7_ERR_INVALID);
                                        CHECK(g_scan.size() == before);
                                        continue;
                                    }
                                    ++accepted;
                                    large += slots * Hv == chunks;
                                    CHECK(wkv7::gdr::prep_blocks(slots, Hv) * 256 < most);
                                    CHECK(wkv7::gdr::grads_blocks(slots, Hk) * 4 * K < most);
                                    // each slab and unit has its place
                                    CHECK(g.slabs * g.groups * 16 >= V && g.slabs * (g.groups - 1) * 16 < V);
                                    CHECK(g.total == seqs * Hv * g.groups && g.blocks >= g.total && g.threads <= 576);
                                }
    CHECK(accepted > 1000 && large > 10);
    // decode has no such launch
    const gdr_shape s{65535, 1, 64, 64, 64, 256, 0, WKV7_BF16, 0, 1.f};
    CHECK(gdr_checkpoint_bytes(&s) == 0);
    CHECK(gdr_decode(&s, kIn, kIn, kIn, kIn, kIn, kIn, 65535, nullptr, kIn, nullptr) == WKV7_OK);
}

// Rows beyond what one launch has threads for.
void many_rows()
{
    const int64_t most = int64_t(1) << 38;
    for (int64_t rows : {int64_t(4194303), int64_t(4194304), int64_t(1) << 32, most, most + 1}) {
        const int ok = rows <= most ? WKV7_OK : WKV7_ERR_UNSUPPORTED;
        for (int64_t D : {1, 1024, 16384}) {
            const residual_norm_shape n{rows, D, WKV7_BF16, 0, 1e-6f};
            const size_t ws = residual_norm_workspace_bytes(&n);
            CHECK((ws > 0) == (ok == WKV7_OK));
            CHECK(residual_norm_forward(&n, kIn, kIn, kIn, kIn, kIn, kIn, nullptr) == ok);
            CHECK(residual_norm_backward(&n, kIn, nullptr, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, ws, nullptr) == ok);
        }
        for (int64_t N : {16, 256}) {
            const gdr_epilogue_shape e{rows, 1, N, 1, WKV7_BF16, 0, 1e-6f};
            const size_t ws = gdr_epilogue_workspace_bytes(&e);
            CHECK((ws > 0) == (ok == WKV7_OK));
            CHECK(gdr_epilogue_forward(&e, kIn, kIn, kIn, kIn, nullptr) == ok);
            CHECK(gdr_epilogue_backward(&e, kIn, kIn, kIn, kIn, kIn, kIn, kIn, kWs, ws, nullptr) == ok);
        }
    }
}
}  // namespace

int main()
{
    oversized();
    edges();
    many_rows();
    return g_fails ? 1 : 0;
}
