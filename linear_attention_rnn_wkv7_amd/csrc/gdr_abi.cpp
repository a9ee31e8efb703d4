// C ABI of the gated delta rule and the residual norm: argument validation,
// workspace layout and dispatch.  Every check runs before anything is
// enqueued on the stream.

#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace {

constexpr size_t kAlign = 256;
// Rows of the norms: more than memory holds.
constexpr int64_t kMaxRows = int64_t(1) << 38;
// Chunks times value heads.
constexpr int64_t kMaxChunks = int64_t(1) << 22;
// Threads of a launch in one dimension stay below 2^32.
constexpr int64_t kMaxThreads = int64_t(1) << 32;

struct Dims {
    int64_t B, T, Hk, Hv, K, V, seqs, nck, slots;
    bool packed, makes;
    int dtype, norm;
    float scale;
    size_t states, rows, table;       // bytes: chunk states, chunk rows, tables
    size_t factors, factors_t;        // of the forward's and the backward's factors, or 0
    int64_t nseg, nckseg;             // segments of a row
    size_t seg_map, carry;            // of the segments, or 0
    bool empty() const { return Hv == 0 || (packed ? seqs == 0 : B == 0); }
    bool tokens() const { return !empty() && B * T > 0; }
};

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

size_t round_up(size_t x);

// Few, long rows run in segments: as many as fill 256 compute units with a
// workgroup each, 16 at most, of at least 4 chunks, where one slab to a
// workgroup would leave units idle (or just fill them).  A chunk then takes two
// steps, one of them with K more columns: fewer than 4 segments do not pay.
void plan_segments(Dims *d)
{
    d->nseg = 1;
    d->nckseg = d->nck;
    const int64_t units = d->B * d->Hv;
    if (d->packed || units == 0 || units * (d->V / 16) > 256) return;
    int64_t n = 256 / units;
    if (n > 16) n = 16;
    if (n > d->nck / 4) n = d->nck / 4;
    if (n < 4) return;
    d->nckseg = (d->nck + n - 1) / n;
    d->nseg = (d->nck + d->nckseg - 1) / d->nckseg;
}

size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void *p) { return ((uintptr_t)p & 15u) == 0; }

int check(const gdr_shape *s, Dims *d)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->B < 0 || s->T < 0 || s->Hk < 0 || s->Hv < 0 || s->K <= 0 || s->V <= 0 || s->nseq < 0)
        return WKV7_ERR_INVALID;
    if (s->dtype != WKV7_F32 && s->dtype != WKV7_BF16) return WKV7_ERR_INVALID;
    if ((s->flags & ~GDR_NORM_QK) != 0) return WKV7_ERR_INVALID;
    if (!std::isnormal(s->scale)) return WKV7_ERR_INVALID;
    if (s->Hk == 0 ? s->Hv != 0 : s->Hv % s->Hk != 0) return WKV7_ERR_INVALID;
    if (s->nseq > 0 && (s->B != 1 || s->T > INT32_MAX)) return WKV7_ERR_INVALID;
    if ((s->K != 64 && s->K != 128) || s->V % 16 != 0 || s->V > 256) return WKV7_ERR_UNSUPPORTED;
    if (s->Hv > 65535) return WKV7_ERR_UNSUPPORTED;
    d->B = s->B;
    d->T = s->T;
    d->Hk = s->Hk;
    d->Hv = s->Hv;
    d->K = s->K;
    d->V = s->V;
    d->packed = s->nseq > 0;
    d->seqs = d->packed ? s->nseq : s->B;
    d->dtype = s->dtype;
    d->norm = (s->flags & GDR_NORM_QK) != 0;
    d->scale = s->scale;
    if (d->seqs > 65535) return WKV7_ERR_UNSUPPORTED;
    const int64_t D = s->K > s->V ? s->K : s->V;
    int64_t x, per;
    // tokens and states of the caller's tensors
    if (!mul_ok(s->B, s->T, &x) || !mul_ok(x, s->Hv + 1, &x) || !mul_ok(x, 4 * D, &x)) return WKV7_ERR_INVALID;
    if (!mul_ok(d->seqs * (s->Hv + 1), s->K * s->V * 4, &x)) return WKV7_ERR_INVALID;
    d->nck = s->T / wkv7::gdr::kChunk + (s->T % wkv7::gdr::kChunk != 0);   // T may be the largest, with B or Hv 0
    if (d->packed)
        d->slots = s->T / wkv7::gdr::kChunk + s->nseq;
    else if (!mul_ok(s->B, d->nck, &d->slots))
        return WKV7_ERR_INVALID;
    if (d->slots > kMaxChunks) return WKV7_ERR_UNSUPPORTED;
    if (!mul_ok(d->slots, s->Hv, &per) || !mul_ok(per, 4 * 4 * (128 * 256 + 64 * 256 + 2 * 4096), &x))
        return WKV7_ERR_INVALID;   // any sum of the workspace's parts
    if (per > kMaxChunks) return WKV7_ERR_UNSUPPORTED;
    plan_segments(d);
    const size_t segs = d->nseg > 1 ? (size_t)(s->B * s->Hv * d->nseg) : 0;
    d->seg_map = segs * (size_t)(s->K * (s->V + s->K) * 4);
    d->carry = segs * (size_t)(s->V * s->K * 4);
    d->states = (size_t)(per * s->K * s->V * 4);
    d->rows = (size_t)(per * 64 * s->V * 4);
    d->makes = wkv7::gdr::scan_makes_factors(d->dtype, s->K, s->V, d->seqs * s->Hv);
    d->factors = d->makes ? 0 : (size_t)per * wkv7::gdr::factor_bytes(d->dtype, false);
    d->factors_t = d->makes ? 0 : (size_t)per * wkv7::gdr::factor_bytes(d->dtype, true);
    d->table = (size_t)(per * wkv7::gdr::kTableFloats * 4);
    return WKV7_OK;
}

// A shape of the chunked calls: every launch of one fits, whichever are made
// (the passes over segments have 256 units at most).
int check_chunked(const gdr_shape *s, Dims *d)
{
    const int rc = check(s, d);
    if (rc != WKV7_OK || !d->tokens()) return rc;
    const wkv7::gdr::ScanGrid g = wkv7::gdr::scan_grid(d->seqs * d->Hv, d->Hv / d->Hk, d->V, d->makes);
    return g.blocks * g.threads < kMaxThreads && wkv7::gdr::prep_blocks(d->slots, d->Hv) * 256 < kMaxThreads &&
                   wkv7::gdr::grads_blocks(d->slots, d->Hk) * 4 * d->K < kMaxThreads
               ? WKV7_OK
               : WKV7_ERR_UNSUPPORTED;
}

size_t segment_bytes(const Dims &d) { return round_up(d.seg_map) + round_up(d.carry); }
size_t forward_bytes(const Dims &d) { return round_up(d.factors) + segment_bytes(d); }
size_t record_bytes(const Dims &d) { return round_up(d.states) + round_up(d.rows); }
// the tables, the factors, the segments, D and dR (sized as the record), and the record if it
// is not given
size_t backward_bytes(const Dims &d, bool ckpt_provided)
{
    return round_up(d.table) + round_up(d.factors_t) + segment_bytes(d) + record_bytes(d) * (ckpt_provided ? 1 : 2);
}

wkv7::gdr::Launch base(const Dims &d, const void *q, const void *k, const void *v, const float *g,
                       const float *beta, const float *s0, const int32_t *starts)
{
    wkv7::gdr::Launch L;
    L.map = {d.packed ? starts : nullptr, d.T, d.seqs, d.nck, d.slots, d.nseg, d.nckseg};
    L.B = d.B;
    L.Hk = d.Hk;
    L.Hv = d.Hv;
    L.K = d.K;
    L.V = d.V;
    L.dtype = d.dtype;
    L.norm = d.norm;
    L.scale = d.scale;
    L.q = q;
    L.k = k;
    L.v = v;
    L.g = g;
    L.beta = beta;
    L.s0 = s0;
    return L;
}

void set_segments(wkv7::gdr::Launch *L, const Dims &d, char *at)
{
    if (d.nseg == 1) return;
    L->seg_map = reinterpret_cast<float *>(at);
    L->carry = reinterpret_cast<float *>(at + round_up(d.seg_map));
}

void set_record(wkv7::gdr::Launch *L, const Dims &d, const float *rec)
{
    char *p = reinterpret_cast<char *>(const_cast<float *>(rec));
    L->rec_s = reinterpret_cast<float *>(p);
    L->rec_e = p ? reinterpret_cast<float *>(p + round_up(d.states)) : nullptr;
}

int status(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP; }

int check_inputs(const Dims &d, std::initializer_list<const void *> needed, std::initializer_list<const void *> maybe,
                 const int32_t *starts)
{
    for (const void *p : needed) {
        if (d.tokens() && !p) return WKV7_ERR_INVALID;
        if (!aligned(p)) return WKV7_ERR_INVALID;
    }
    for (const void *p : maybe)
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (d.packed != (starts != nullptr) || !aligned(starts)) return WKV7_ERR_INVALID;
    return WKV7_OK;
}

int check_workspace(const void *ws, size_t given, size_t need)
{
    if (need == 0) return WKV7_OK;
    return ws && given >= need && (uintptr_t)ws % kAlign == 0 ? WKV7_OK : WKV7_ERR_WORKSPACE;
}

int check(const gdr_epilogue_shape *s, wkv7::gdr::EpilogueLaunch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->rows < 0 || s->H < 0 || s->N <= 0 || s->flags != 0) return WKV7_ERR_INVALID;
    if (s->dtype != WKV7_F32 && s->dtype != WKV7_BF16) return WKV7_ERR_INVALID;
    if (!(s->eps > 0.f) || !isfinite(s->eps)) return WKV7_ERR_INVALID;
    if (s->Hw != 1 && s->Hw != s->H) return WKV7_ERR_INVALID;
    if (s->N < 16 || s->N > 256 || (s->N & (s->N - 1)) != 0 || s->Hw > 65535) return WKV7_ERR_UNSUPPORTED;
    int64_t n, x;
    if (!mul_ok(s->rows, s->H, &n) || !mul_ok(n, s->N * 4, &x)) return WKV7_ERR_INVALID;
    if (n > kMaxRows) return WKV7_ERR_UNSUPPORTED;
    L->rows = s->rows;
    L->H = s->H;
    L->N = s->N;
    L->Hw = s->Hw;
    L->dtype = s->dtype;
    L->eps = s->eps;
    return WKV7_OK;
}

int check(const residual_norm_shape *s, wkv7::gdr::NormLaunch *L)
{
    if (!s) return WKV7_ERR_INVALID;
    if (s->rows < 0 || s->D <= 0 || s->flags != 0) return WKV7_ERR_INVALID;
    if (s->dtype != WKV7_F32 && s->dtype != WKV7_BF16) return WKV7_ERR_INVALID;
    if (!(s->eps > 0.f) || !isfinite(s->eps)) return WKV7_ERR_INVALID;
    if (s->D > 16384) return WKV7_ERR_UNSUPPORTED;
    if (s->rows > kMaxRows) return WKV7_ERR_UNSUPPORTED;
    L->rows = s->rows;
    L->D = s->D;
    L->dtype = s->dtype;
    L->eps = s->eps;
    return WKV7_OK;
}

size_t parts_bytes(const wkv7::gdr::EpilogueLaunch &L)
{
    if (L.rows * L.H == 0) return 0;
    return round_up((size_t)(L.Hw * wkv7::gdr::epilogue_parts(L.rows, L.H, L.N, L.Hw) * L.N) * sizeof(float));
}

size_t parts_bytes(const wkv7::gdr::NormLaunch &L)
{
    return L.rows == 0 ? 0 : round_up((size_t)(wkv7::gdr::norm_parts(L.rows, L.D) * 2 * L.D) * sizeof(float));
}

}  // namespace

extern "C" {

size_t gdr_checkpoint_bytes(const gdr_shape *shape)
{
    Dims d;
    if (check_chunked(shape, &d) != WKV7_OK || !d.tokens()) return 0;
    return record_bytes(d);
}

size_t gdr_forward_workspace_bytes(const gdr_shape *shape)
{
    Dims d;
    if (check_chunked(shape, &d) != WKV7_OK || !d.tokens()) return 0;
    return forward_bytes(d);
}

size_t gdr_backward_workspace_bytes(const gdr_shape *shape, int ckpt_provided)
{
    Dims d;
    if (check_chunked(shape, &d) != WKV7_OK || !d.tokens()) return 0;
    return backward_bytes(d, ckpt_provided != 0);
}

int gdr_forward(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
                const float *beta, const float *s0, const int32_t *seq_starts, void *y, float *sT,
                float *ckpt, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    Dims d;
    int rc = check_chunked(shape, &d);
    if (rc != WKV7_OK) return rc;
    rc = check_inputs(d, {q, k, v, g, beta}, {s0, y, sT, ckpt}, seq_starts);
    if (rc != WKV7_OK) return rc;
    if (d.empty()) return WKV7_OK;
    if (!d.tokens()) {
        if (!sT) return WKV7_OK;
        return status(wkv7::launch_fill(sT, s0, (size_t)(d.seqs * d.Hv * d.K * d.V), stream));
    }
    rc = check_workspace(workspace, workspace_bytes, forward_bytes(d));
    if (rc != WKV7_OK) return rc;
    wkv7::gdr::Launch L = base(d, q, k, v, g, beta, s0, seq_starts);
    L.factors = d.factors ? workspace : nullptr;
    set_segments(&L, d, static_cast<char *>(workspace) + round_up(d.factors));
    L.y = y;
    L.sT = sT;
    set_record(&L, d, ckpt);
    if (!y && !sT && !ckpt) return WKV7_OK;
    return status(wkv7::gdr::launch_scan(L, stream));
}

int gdr_backward(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
                 const float *beta, const float *s0, const int32_t *seq_starts, const void *dy,
                 const float *dsT, const float *ckpt, void *dq, void *dk, void *dv, float *dg,
                 float *dbeta, float *ds0, void *workspace, size_t workspace_bytes,
                 hipStream_t stream)
{
    Dims d;
    int rc = check_chunked(shape, &d);
    if (rc != WKV7_OK) return rc;
    rc = check_inputs(d, {q, k, v, g, beta, dy, dq, dk, dv, dg, dbeta}, {s0, dsT, ckpt, ds0}, seq_starts);
    if (rc != WKV7_OK) return rc;
    if (d.empty()) return WKV7_OK;
    if (!d.tokens()) {
        if (!ds0) return WKV7_OK;
        return status(wkv7::launch_fill(ds0, dsT, (size_t)(d.seqs * d.Hv * d.K * d.V), stream));
    }
    rc = check_workspace(workspace, workspace_bytes, backward_bytes(d, ckpt != nullptr));
    if (rc != WKV7_OK) return rc;
    char *ws = static_cast<char *>(workspace), *segs = ws + round_up(d.table) + round_up(d.factors_t),
         *grads = segs + segment_bytes(d);
    wkv7::gdr::Launch L = base(d, q, k, v, g, beta, s0, seq_starts);
    L.table = static_cast<float *>(workspace);
    L.factors = d.factors_t ? ws + round_up(d.table) : nullptr;   // at least the forward's
    set_segments(&L, d, segs);
    L.ws_ds = reinterpret_cast<float *>(grads);
    L.ws_dr = reinterpret_cast<float *>(grads + round_up(d.states));
    if (ckpt) {
        set_record(&L, d, ckpt);
    } else {
        set_record(&L, d, reinterpret_cast<const float *>(grads + record_bytes(d)));
        rc = status(wkv7::gdr::launch_scan(L, stream));
        if (rc != WKV7_OK) return rc;
    }
    L.dy = dy;
    L.dsT = dsT;
    L.dq = dq;
    L.dk = dk;
    L.dv = dv;
    L.dg = dg;
    L.dbeta = dbeta;
    L.ds0 = ds0;
    rc = status(wkv7::gdr::launch_reverse(L, stream));
    if (rc == WKV7_OK) rc = status(wkv7::gdr::launch_grads(L, stream));
    return rc;
}

int gdr_decode(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
               const float *beta, float *state, int64_t pool, const int32_t *slots, void *y,
               hipStream_t stream)
{
    Dims d;
    int rc = check(shape, &d);
    if (rc != WKV7_OK) return rc;
    if (d.packed || pool < 0 || (!slots && pool < d.B) || pool > INT32_MAX) return WKV7_ERR_INVALID;
    int64_t x;
    if (!mul_ok(pool, (d.Hv + 1) * d.K * d.V * 4, &x)) return WKV7_ERR_INVALID;
    for (const void *p : {q, k, v, (const void *)g, (const void *)beta, (const void *)state, (const void *)y}) {
        if (d.tokens() && pool > 0 && !p) return WKV7_ERR_INVALID;
        if (!aligned(p)) return WKV7_ERR_INVALID;
    }
    if (!aligned(slots)) return WKV7_ERR_INVALID;
    if (!d.tokens() || pool == 0) return WKV7_OK;
    wkv7::gdr::DecodeLaunch L = {d.B, d.T, d.Hk, d.Hv, d.K, d.V, pool, d.dtype, d.norm, d.scale,
                                 q, k, v, g, beta, state, slots, y};
    return status(wkv7::gdr::launch_decode(L, stream));
}

size_t gdr_epilogue_workspace_bytes(const gdr_epilogue_shape *shape)
{
    wkv7::gdr::EpilogueLaunch L;
    return check(shape, &L) == WKV7_OK ? parts_bytes(L) : 0;
}

int gdr_epilogue_forward(const gdr_epilogue_shape *shape, const void *y, const void *gate,
                         const float *w, void *z, hipStream_t stream)
{
    wkv7::gdr::EpilogueLaunch L;
    const int rc = check(shape, &L);
    if (rc != WKV7_OK) return rc;
    if (L.rows * L.H == 0) return WKV7_OK;
    for (const void *p : {y, gate, (const void *)w, (const void *)z})
        if (!p || !aligned(p)) return WKV7_ERR_INVALID;
    L.y = y;
    L.gate = gate;
    L.w = w;
    L.z = z;
    return status(wkv7::gdr::launch_epilogue_forward(L, stream));
}

int gdr_epilogue_backward(const gdr_epilogue_shape *shape, const void *dz, const void *y,
                          const void *gate, const float *w, void *dy, void *dgate, float *dw,
                          void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    wkv7::gdr::EpilogueLaunch L;
    int rc = check(shape, &L);
    if (rc != WKV7_OK) return rc;
    if (L.Hw == 0) return WKV7_OK;
    if (!dw || !aligned(dw)) return WKV7_ERR_INVALID;
    if (L.rows * L.H == 0) return status(wkv7::launch_fill(dw, nullptr, (size_t)(L.Hw * L.N), stream));
    for (const void *p : {dz, y, gate, (const void *)w, (const void *)dy, (const void *)dgate})
        if (!p || !aligned(p)) return WKV7_ERR_INVALID;
    rc = check_workspace(workspace, workspace_bytes, parts_bytes(L));
    if (rc != WKV7_OK) return rc;
    L.dz = dz;
    L.y = y;
    L.gate = gate;
    L.w = w;
    L.dy = dy;
    L.dgate = dgate;
    L.dw = dw;
    L.part = static_cast<float *>(workspace);
    return status(wkv7::gdr::launch_epilogue_backward(L, stream));
}

size_t residual_norm_workspace_bytes(const residual_norm_shape *shape)
{
    wkv7::gdr::NormLaunch L;
    return check(shape, &L) == WKV7_OK ? parts_bytes(L) : 0;
}

int residual_norm_forward(const residual_norm_shape *shape, const void *x, const void *y,
                          const float *scale, const float *w, void *x_out, void *h,
                          hipStream_t stream)
{
    wkv7::gdr::NormLaunch L;
    const int rc = check(shape, &L);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {x, y, (const void *)scale, (const void *)w, (const void *)x_out, (const void *)h})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (L.rows == 0) return WKV7_OK;
    if (!x || !w || !h || (scale && !y)) return WKV7_ERR_INVALID;
    L.x = x;
    L.y = y;
    L.scale = scale;
    L.w = w;
    L.x_out = x_out;
    L.h = h;
    return status(wkv7::gdr::launch_norm_forward(L, stream));
}

int residual_norm_backward(const residual_norm_shape *shape, const void *dh, const void *dx_out,
                           const void *x_out, const void *y, const float *scale, const float *w,
                           void *dx, void *dy, float *dw, float *dscale, void *workspace,
                           size_t workspace_bytes, hipStream_t stream)
{
    wkv7::gdr::NormLaunch L;
    int rc = check(shape, &L);
    if (rc != WKV7_OK) return rc;
    for (const void *p : {dh, dx_out, x_out, y, (const void *)scale, (const void *)w, (const void *)dx,
                          (const void *)dy, (const void *)dw, (const void *)dscale})
        if (!aligned(p)) return WKV7_ERR_INVALID;
    if (!dw) return WKV7_ERR_INVALID;
    if ((scale != nullptr) != (dscale != nullptr)) return WKV7_ERR_INVALID;
    if (L.rows == 0) {
        rc = status(wkv7::launch_fill(dw, nullptr, (size_t)L.D, stream));
        if (rc == WKV7_OK && dscale) rc = status(wkv7::launch_fill(dscale, nullptr, (size_t)L.D, stream));
        return rc;
    }
    if (!dh || !x_out || !w || !dx) return WKV7_ERR_INVALID;
    if ((scale != nullptr) != (y != nullptr) || (scale != nullptr) != (dy != nullptr)) return WKV7_ERR_INVALID;
    rc = check_workspace(workspace, workspace_bytes, parts_bytes(L));
    if (rc != WKV7_OK) return rc;
    L.dh = dh;
    L.dx_out = dx_out;
    L.x_out = const_cast<void *>(x_out);
    L.y = y;
    L.scale = scale;
    L.w = w;
    L.dx = dx;
    L.dy = dy;
    L.dw = dw;
    L.dscale = dscale;
    L.part = static_cast<float *>(workspace);
    return status(wkv7::gdr::launch_norm_backward(L, stream));
}

}  // extern "C"
