// The scans over the chunks, forward and reverse (the mathematics and the
// operand layouts: gdr_device.h).
//
// One wave owns 16 value columns of one sequence's head: its K x 16 slab of
// the state stays in registers as result tiles, and every product of the
// chain takes its other operand from LDS, so that a chunk needs no exchange
// between waves.  The waves of a workgroup share that operand: K and Q by
// rows, K (and in the reverse scan Q) transposed, and the chunk's triangular
// factors.
//
// Reverse, from the gradient D of the state behind the chunk:
//     dE = P^T dY + w * (K D),  w_j = (gamma_C / gamma_j) beta_j
//     dR = T^T dE  (= dV)
//     D0 = gamma_C D + (gamma Q)^T dY - (gamma K)^T dR
// It leaves D (per chunk) and dR for gdr_grads.hip.

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {
namespace {

template <typename T>
struct ScanArgs {
    Map map;
    const T *q, *k, *v, *dy;
    const float *s0, *dsT;
    T *y, *dv;
    float *sT, *ds0;
    float *st, *rows;    // record: states and E; reverse: D and dR
    const float *table;
    const T *tfrag, *pfrag;
    int64_t Hk, Hv, V;
    int group;
};

// Rows of [64][K] (stride Hk * K in memory) into LDS by rows and transposed.
template <typename T, int K, bool kRows, bool kCols>
__device__ __forceinline__ void stage(const T *src, int64_t stride, int len, T *rows, T *cols, int tid, int nt)
{
    using Quad = typename Num<T>::Quad;
    constexpr int LD = K + kPad<T>, LT = 64 + kPad<T>;
    for (int b = tid; b < 16 * (K / 4); b += nt) {
        const int col = 4 * (b % (K / 4)), t0 = 4 * (b / (K / 4));
        Quad x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = Quad{};
            if (t0 + r < len) x[r] = *reinterpret_cast<const Quad *>(src + (t0 + r) * stride + col);
        }
        if constexpr (kRows) {
#pragma unroll
            for (int r = 0; r < 4; ++r) *reinterpret_cast<Quad *>(rows + (t0 + r) * LD + kpos(col)) = x[r];
        }
        if constexpr (kCols) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Quad z = {x[0][i], x[1][i], x[2][i], x[3][i]};
                *reinterpret_cast<Quad *>(cols + (col + i) * LT + kpos(t0)) = z;
            }
        }
    }
}

// A chunk's fragments and table rows into LDS.
template <typename T>
__device__ __forceinline__ void stage_frags(const T *src, T *dst, int tid, int nt)
{
    using Oct = typename Num<T>::Oct;
    for (int i = tid; i < Num<T>::kPlanes * kFragElems / 8; i += nt)
        reinterpret_cast<Oct *>(dst)[i] = reinterpret_cast<const Oct *>(src)[i];
}

template <typename T, int K>
struct FwdLds {
    T k[64 * (K + kPad<T>)], q[64 * (K + kPad<T>)], kt[K * (64 + kPad<T>)];
    T t[Num<T>::kPlanes * kFragElems], p[Num<T>::kPlanes * kFragElems];
    float tab[8 * 64];
};

template <typename T, int K, bool kY>
__global__ void __launch_bounds__(512) gdr_scan_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes, LD = K + kPad<T>, LT = 64 + kPad<T>;
    constexpr int KT = K / 16, KS = K / 32;
    __shared__ __align__(16) char buf[sizeof(FwdLds<T, K>)];
    FwdLds<T, K> &s = *reinterpret_cast<FwdLds<T, K> *>(buf);
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, lg = lane >> 4, l16 = lane & 15;
    const int64_t seq = blockIdx.z, hv = blockIdx.y, hk = hv / a.group;
    const int64_t col = 16 * ((int64_t)blockIdx.x * (nt >> 6) + (tid >> 6)) + l16;
    const bool own = col < a.V;   // whole waves
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;

    f32x4 S[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        S[i] = a.s0 && own ? *reinterpret_cast<const f32x4 *>(a.s0 + so + 16 * i) : zero4();

    for (int64_t c = 0; c < nc; ++c) {
        const int64_t tok = lo + c * kChunk, ch = (slot0 + c) * a.Hv + hv;
        const int len = hi - tok < kChunk ? (int)(hi - tok) : kChunk;
        __syncthreads();   // the previous chunk's operands are done with
        stage<T, K, true, true>(a.k + (tok * a.Hk + hk) * K, a.Hk * K, len, s.k, s.kt, tid, nt);
        if constexpr (kY) {
            stage<T, K, true, false>(a.q + (tok * a.Hk + hk) * K, a.Hk * K, len, s.q, nullptr, tid, nt);
            stage_frags(a.pfrag + ch * P * kFragElems, s.p, tid, nt);
        }
        stage_frags(a.tfrag + ch * P * kFragElems, s.t, tid, nt);
        for (int i = tid; i < kTableFloats / 4; i += nt)
            reinterpret_cast<f32x4 *>(s.tab)[i] = reinterpret_cast<const f32x4 *>(a.table + ch * kTableFloats)[i];
        f32x4 R[4];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * it + 4 * lg + r;
                R[it][r] = own && t < len ? to_f32(a.v[((tok + t) * a.Hv + hv) * a.V + col]) : 0.f;
            }
        __syncthreads();
        if (!own) continue;
        if (a.st) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a.st[(ch * K + 16 * i + 4 * lg + r) * a.V + col] = S[i][r];
        }
        Frag<T, P> Sf[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) Sf[ks] = make_frag<T, P>(S[2 * ks], S[2 * ks + 1]);
        f32x4 Y[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f32x4 acc = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                acc = mma(acc, load_frag<T, 1>(s.k, 16 * it + l16, LD, ks, lg, 0), Sf[ks]);
            R[it] -= row4(s.tab, 0, 16 * it + 4 * lg) * acc;
            if constexpr (kY) {
                acc = zero4();
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    acc = mma(acc, load_frag<T, 1>(s.q, 16 * it + l16, LD, ks, lg, 0), Sf[ks]);
                Y[it] = row4(s.tab, 1, 16 * it + 4 * lg) * acc;
            }
        }
        const Frag<T, P> Rf[2] = {make_frag<T, P>(R[0], R[1]), make_frag<T, P>(R[2], R[3])};
        f32x4 E[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            E[it] = zero4();
#pragma unroll
            for (int ks = 0; ks <= it / 2; ++ks)
                E[it] = mma(E[it], load_packed<T, P>(s.t, low_frag(it, ks), lane), Rf[ks]);
            if (a.rows) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a.rows[(ch * 64 + 16 * it + 4 * lg + r) * a.V + col] = E[it][r];
            }
        }
        if constexpr (kY) {
            const Frag<T, P> Ef[2] = {make_frag<T, P>(E[0], E[1]), make_frag<T, P>(E[2], E[3])};
#pragma unroll
            for (int it = 0; it < 4; ++it) {
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks)
                    Y[it] = mma(Y[it], load_packed<T, P>(s.p, low_frag(it, ks), lane), Ef[ks]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * it + 4 * lg + r;
                    if (t < len) a.y[((tok + t) * a.Hv + hv) * a.V + col] = (T)Y[it][r];
                }
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) E[it] *= row4(s.tab, 2, 16 * it + 4 * lg);
        const Frag<T, P> Wf[2] = {make_frag<T, P>(E[0], E[1]), make_frag<T, P>(E[2], E[3])};
        const float last = expf(s.tab[4 * 64 + 63]);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            S[i] *= last;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                S[i] = mma(S[i], load_frag<T, 1>(s.kt, 16 * i + l16, LT, ks, lg, 0), Wf[ks]);
        }
    }
    if (a.sT && own) {
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(a.sT + so + 16 * i) = S[i];
    }
}

template <typename T, int K>
struct RevLds {
    T k[64 * (K + kPad<T>)], kt[K * (64 + kPad<T>)], qt[K * (64 + kPad<T>)];
    T t[Num<T>::kPlanes * kFragElems], p[Num<T>::kPlanes * kFragElems];
    float tab[8 * 64];
};

template <typename T, int K>
__global__ void __launch_bounds__(512) gdr_reverse_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes, LD = K + kPad<T>, LT = 64 + kPad<T>;
    constexpr int KT = K / 16, KS = K / 32;
    __shared__ __align__(16) char buf[sizeof(RevLds<T, K>)];
    RevLds<T, K> &s = *reinterpret_cast<RevLds<T, K> *>(buf);
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, lg = lane >> 4, l16 = lane & 15;
    const int64_t seq = blockIdx.z, hv = blockIdx.y, hk = hv / a.group;
    const int64_t col = 16 * ((int64_t)blockIdx.x * (nt >> 6) + (tid >> 6)) + l16;
    const bool own = col < a.V;
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;

    f32x4 D[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        D[i] = a.dsT && own ? *reinterpret_cast<const f32x4 *>(a.dsT + so + 16 * i) : zero4();

    for (int64_t c = nc - 1; c >= 0; --c) {
        const int64_t tok = lo + c * kChunk, ch = (slot0 + c) * a.Hv + hv;
        const int len = hi - tok < kChunk ? (int)(hi - tok) : kChunk;
        __syncthreads();
        stage<T, K, true, true>(a.k + (tok * a.Hk + hk) * K, a.Hk * K, len, s.k, s.kt, tid, nt);
        stage<T, K, false, true>(a.q + (tok * a.Hk + hk) * K, a.Hk * K, len, nullptr, s.qt, tid, nt);
        stage_frags(a.pfrag + ch * P * kFragElems, s.p, tid, nt);
        stage_frags(a.tfrag + ch * P * kFragElems, s.t, tid, nt);
        for (int i = tid; i < kTableFloats / 4; i += nt)
            reinterpret_cast<f32x4 *>(s.tab)[i] = reinterpret_cast<const f32x4 *>(a.table + ch * kTableFloats)[i];
        f32x4 dY[4];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * it + 4 * lg + r;
                dY[it][r] = own && t < len ? to_f32(a.dy[((tok + t) * a.Hv + hv) * a.V + col]) : 0.f;
            }
        __syncthreads();
        if (!own) continue;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                a.st[(ch * K + 16 * i + 4 * lg + r) * a.V + col] = D[i][r];
        Frag<T, P> Df[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) Df[ks] = make_frag<T, P>(D[2 * ks], D[2 * ks + 1]);
        const Frag<T, 1> dYf[2] = {make_frag<T, 1>(dY[0], dY[1]), make_frag<T, 1>(dY[2], dY[3])};
        f32x4 dE[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            f32x4 acc = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                acc = mma(acc, load_frag<T, 1>(s.k, 16 * jt + l16, LD, ks, lg, 0), Df[ks]);
            dE[jt] = row4(s.tab, 2, 16 * jt + 4 * lg) * acc;
#pragma unroll
            for (int ks = jt / 2; ks < 2; ++ks)
                dE[jt] = mma(dE[jt], load_packed<T, P>(s.p, up_frag(jt, ks), lane), dYf[ks]);
        }
        const Frag<T, P> dEf[2] = {make_frag<T, P>(dE[0], dE[1]), make_frag<T, P>(dE[2], dE[3])};
        f32x4 dR[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            dR[jt] = zero4();
#pragma unroll
            for (int ks = jt / 2; ks < 2; ++ks)
                dR[jt] = mma(dR[jt], load_packed<T, P>(s.t, up_frag(jt, ks), lane), dEf[ks]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * jt + 4 * lg + r;
                a.rows[(ch * 64 + t) * a.V + col] = dR[jt][r];
                if (t < len) a.dv[((tok + t) * a.Hv + hv) * a.V + col] = (T)dR[jt][r];
            }
            dY[jt] *= row4(s.tab, 1, 16 * jt + 4 * lg);
            dR[jt] *= -row4(s.tab, 0, 16 * jt + 4 * lg);
        }
        const Frag<T, P> Yf[2] = {make_frag<T, P>(dY[0], dY[1]), make_frag<T, P>(dY[2], dY[3])};
        const Frag<T, P> Rf[2] = {make_frag<T, P>(dR[0], dR[1]), make_frag<T, P>(dR[2], dR[3])};
        const float last = expf(s.tab[4 * 64 + 63]);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            D[i] *= last;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                D[i] = mma(D[i], load_frag<T, 1>(s.qt, 16 * i + l16, LT, ks, lg, 0), Yf[ks]);
                D[i] = mma(D[i], load_frag<T, 1>(s.kt, 16 * i + l16, LT, ks, lg, 0), Rf[ks]);
            }
        }
    }
    if (a.ds0 && own) {
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(a.ds0 + so + 16 * i) = D[i];
    }
}

template <typename T>
ScanArgs<T> scan_args(const Launch &a)
{
    ScanArgs<T> p;
    p.map = a.map;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.v = static_cast<const T *>(a.v);
    p.dy = static_cast<const T *>(a.dy);
    p.s0 = a.s0;
    p.dsT = a.dsT;
    p.y = static_cast<T *>(a.y);
    p.dv = static_cast<T *>(a.dv);
    p.sT = a.sT;
    p.ds0 = a.ds0;
    p.st = a.rec_s;
    p.rows = a.rec_e;
    p.table = a.table;
    p.tfrag = static_cast<const T *>(a.tfrag);
    p.pfrag = static_cast<const T *>(a.pfrag);
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.V = a.V;
    p.group = (int)(a.Hv / a.Hk);
    return p;
}

// Slabs per workgroup: as many as there are (8 at most), fewer while that
// leaves compute units without a workgroup.
void scan_grid(const Launch &a, dim3 *grid, dim3 *block)
{
    const int64_t slabs = a.V / 16, units = a.map.nseq * a.Hv;
    int64_t groups = (slabs + 7) / 8;
    while (units * groups < 256 && groups < slabs) ++groups;
    const int64_t per = (slabs + groups - 1) / groups;
    *grid = dim3((unsigned)((slabs + per - 1) / per), (unsigned)a.Hv, (unsigned)a.map.nseq);
    *block = dim3((unsigned)(64 * per));
}

template <typename T, int K>
hipError_t scan_t(const Launch &a, bool reverse, hipStream_t stream)
{
    ScanArgs<T> p = scan_args<T>(a);
    dim3 grid, block;
    scan_grid(a, &grid, &block);
    if (reverse) {
        p.st = a.ws_ds;
        p.rows = a.ws_dr;
        hipLaunchKernelGGL((gdr_reverse_kernel<T, K>), grid, block, 0, stream, p);
    } else if (a.y) {
        hipLaunchKernelGGL((gdr_scan_kernel<T, K, true>), grid, block, 0, stream, p);
    } else {
        hipLaunchKernelGGL((gdr_scan_kernel<T, K, false>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

hipError_t scan_any(const Launch &a, bool reverse, hipStream_t stream)
{
    if (a.dtype == WKV7_F32)
        return a.K == 64 ? scan_t<float, 64>(a, reverse, stream) : scan_t<float, 128>(a, reverse, stream);
    return a.K == 64 ? scan_t<bf16, 64>(a, reverse, stream) : scan_t<bf16, 128>(a, reverse, stream);
}

}  // namespace

hipError_t launch_scan(const Launch &a, hipStream_t stream) { return scan_any(a, false, stream); }
hipError_t launch_reverse(const Launch &a, hipStream_t stream) { return scan_any(a, true, stream); }

}  // namespace gdr
}  // namespace wkv7
