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

// The lane's first row and column in a wave's tiles, fresh to the compiler at
// each use: otherwise it keeps every offset made from it in a register.
__device__ __forceinline__ uint32_t fresh(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// A wave's 64 x 16 tiles of a chunk of a [tokens][Hv][V] tensor, by buffer
// accesses: rows behind the chunk's last read as zero and are not written.
template <typename T>
struct Cols {
    BufRsrc buf;
    uint32_t at, step;   // this lane's first row and column; bytes of a token

    __device__ __forceinline__ Cols(const T *base, int64_t stride, int64_t V, int64_t col, int len, int lg)
        : buf(raw_buffer(base, (uint32_t)(((len - 1) * stride + V) * (int64_t)sizeof(T)))),
          at(fresh((uint32_t)((4 * lg * stride + col) * (int64_t)sizeof(T)))), step((uint32_t)(stride * (int64_t)sizeof(T)))
    {
    }
    __device__ __forceinline__ uint32_t off(int i) const { return at + (16 * (i >> 2) + (i & 3)) * step; }
    __device__ __forceinline__ T load(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buf, (int)off(i), 0, 0));
        else
            return __builtin_bit_cast(T, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(buf, (int)off(i), 0, 0));
    }
    __device__ __forceinline__ void store(int i, float x) const
    {
        if constexpr (sizeof(T) == 4)
            bstore(buf, off(i), x);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (T)x), buf, (int)off(i), 0, 0);
    }
};

// Whole 16-row tiles i of a [rows][V] fp32 matrix.
struct Tiles {
    BufRsrc buf;
    uint32_t at, step;

    __device__ __forceinline__ Tiles(float *base, int rows, int64_t V, int64_t col, int lg)
        : buf(raw_buffer(base, (uint32_t)(rows * V * 4))), at(fresh((uint32_t)((4 * lg * V + col) * 4))), step((uint32_t)(V * 4))
    {
    }
    __device__ __forceinline__ void store(int i, f32x4 x) const
    {
#pragma unroll
        for (int r = 0; r < 4; ++r) bstore(buf, at + (16 * i + r) * step, x[r]);
    }
};

// Where a workgroup stands in its sequence.
struct Pos {
    int64_t tok, ch;
    int len;
};
__device__ __forceinline__ Pos chunk_at(int64_t lo, int64_t hi, int64_t slot0, int64_t c, int64_t Hv, int64_t hv)
{
    const int64_t tok = lo + c * kChunk;
    return {tok, (slot0 + c) * Hv + hv, hi - tok < kChunk ? (int)(hi - tok) : kChunk};
}

// One chunk's operands in LDS.  The copies of the next chunk run while this
// one is computed, into a second set, where two fit into 160 KB (all but
// fp32 with K = 128).
template <typename T, int K, int PP>
struct Operands {
    static constexpr int kMat = Swizzled<T, K>::kBytes;
    static constexpr int kT = Num<T>::kPlanes * kFragElems * (int)sizeof(T), kP = PP * kFragElems * (int)sizeof(T);
    static constexpr int kTab = kTableFloats * 4;
    static constexpr int kBytes = 2 * kMat + kT + kP + kTab;
    static constexpr int kSets = 2 * kBytes <= 160 * 1024 ? 2 : 1;
    char *base;

    __device__ __forceinline__ char *k() const { return base; }
    __device__ __forceinline__ char *q() const { return base + kMat; }
    __device__ __forceinline__ const T *t() const { return reinterpret_cast<const T *>(base + 2 * kMat); }
    __device__ __forceinline__ const T *p() const { return reinterpret_cast<const T *>(base + 2 * kMat + kT); }
    __device__ __forceinline__ const float *tab() const
    {
        return reinterpret_cast<const float *>(base + 2 * kMat + kT + kP);
    }
    template <bool kAll>
    __device__ __forceinline__ void copy(const ScanArgs<T> &a, const Pos &at, int64_t hk, int lane) const
    {
        const int64_t o = (at.tok * a.Hk + hk) * K;
        dma_rows<T, K>(k(), a.k + o, a.Hk * K, at.len, lane);
        dma_flat<kT>(base + 2 * kMat, a.tfrag + at.ch * (kT / (int)sizeof(T)), lane);
        dma_flat<kTab>(base + 2 * kMat + kT + kP, a.table + at.ch * kTableFloats, lane);
        if constexpr (kAll) {
            dma_rows<T, K>(q(), a.q + o, a.Hk * K, at.len, lane);
            dma_flat<kP>(base + 2 * kMat + kT, a.pfrag + at.ch * (kP / (int)sizeof(T)), lane);
        }
    }
};

template <typename T, int P, int Q>
__device__ __forceinline__ Frag<T, Q> first_parts(const Frag<T, P> &f)
{
    Frag<T, Q> g;
#pragma unroll
    for (int i = 0; i < Q; ++i) g.p[i] = f.p[i];
    return g;
}

// The last wave of a workgroup copies the operands, chunk by chunk, one ahead
// of the others: issuing copies stalls whenever the memory system has no room
// for more, and would stall the products with it.  One barrier per chunk: the
// copies for it have landed, and the set of the chunk before is free.
template <typename T, int K, int PP, bool kAll>
__device__ __forceinline__ void copy_loop(const ScanArgs<T> &a, char *buf, int64_t lo, int64_t hi, int64_t slot0,
                                          int64_t hv, int64_t hk, int64_t first, int64_t step, int64_t nc, int lane)
{
    using Op = Operands<T, K, PP>;
    __builtin_amdgcn_s_setprio(2);
    for (int64_t i = 0, c = first; i < nc; ++i, c += step) {
        if (Op::kSets == 1 && i > 0) __syncthreads();   // the only set is free
        Op{buf + (Op::kSets == 2 ? (i & 1) * Op::kBytes : 0)}.template copy<kAll>(
            a, chunk_at(lo, hi, slot0, c, a.Hv, hv), hk, lane);
        wait_dma();
        __syncthreads();
    }
}

constexpr int kMaxThreads = 64 * 9;   // 8 slabs and the copies

template <typename T, int K, bool kY>
__global__ void __launch_bounds__(kMaxThreads) gdr_scan_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes, PY = kYParts<T>;
    constexpr int KT = K / 16, KS = K / 32;
    using Op = Operands<T, K, PY>;
    using Sw = Swizzled<T, K>;
    __shared__ __align__(16) char buf[Op::kSets * Op::kBytes];
    const int lane = threadIdx.x & 63, lg = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), slabs = (blockDim.x >> 6) - 1;
    const int64_t seq = blockIdx.z, hv = blockIdx.y, hk = hv / a.group;
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;
    if (wave == slabs) {
        copy_loop<T, K, PY, kY>(a, buf, lo, hi, slot0, hv, hk, 0, 1, nc, lane);
        return;
    }
    const int64_t col = 16 * ((int64_t)blockIdx.x * slabs + wave) + l16;
    const bool own = 16 * ((int64_t)blockIdx.x * slabs + wave) < a.V;

    f32x4 S[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        S[i] = a.s0 && own ? *reinterpret_cast<const f32x4 *>(a.s0 + so + 16 * i) : zero4();

    T vn[16];
    auto fetch = [&](int64_t c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Cols<T> v(a.v + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
        for (int i = 0; i < 16; ++i) vn[i] = v.load(i);
    };
    if (own && nc > 0) fetch(0);
    for (int64_t c = 0; c < nc; ++c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Op s{buf + (Op::kSets == 2 ? (c & 1) * Op::kBytes : 0)};
        __syncthreads();
        if (own) {
            f32x4 R[4], Y[4];
#pragma unroll
            for (int i = 0; i < 16; ++i) R[i >> 2][i & 3] = to_f32(vn[i]);
            if (c + 1 < nc) fetch(c + 1);
            if (a.st) {
                const Tiles st(a.st + at.ch * K * a.V, K, a.V, col, lg);
#pragma unroll
                for (int i = 0; i < KT; ++i) st.store(i, S[i]);
            }
            {   // K S and Q S
                f32x4 acc[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) acc[it] = Y[it] = zero4();
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const Frag<T, P> Sf = make_frag<T, P>(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        acc[it] = mma(acc[it], Sw::rows(s.k(), it, ks, lg, l16), Sf);
                        if constexpr (kY)
                            Y[it] = mma<PY>(Y[it], Sw::rows(s.q(), it, ks, lg, l16), first_parts<T, P, PY>(Sf));
                    }
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) R[it] -= row4(s.tab(), 0, 16 * it + 4 * lg) * acc[it];
            }
            const Frag<T, P> Rf[2] = {make_frag<T, P>(R[0], R[1]), make_frag<T, P>(R[2], R[3])};
            f32x4 E[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                E[it] = zero4();
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks)
                    E[it] = mma(E[it], load_packed<T, P>(s.t(), low_frag(it, ks), lane), Rf[ks]);
            }
            if (a.rows) {
                const Tiles rows(a.rows + at.ch * 64 * a.V, 64, a.V, col, lg);
#pragma unroll
                for (int i = 0; i < 4; ++i) rows.store(i, E[i]);
            }
            if constexpr (kY) {
                const Frag<T, PY> Ef[2] = {make_frag<T, PY>(E[0], E[1]), make_frag<T, PY>(E[2], E[3])};
                const Cols<T> y(a.y + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    Y[it] *= row4(s.tab(), 1, 16 * it + 4 * lg);
#pragma unroll
                    for (int ks = 0; ks <= it / 2; ++ks)
                        Y[it] = mma<PY>(Y[it], load_packed<T, PY>(s.p(), low_frag(it, ks), lane), Ef[ks]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y.store(4 * it + r, Y[it][r]);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) E[it] *= row4(s.tab(), 2, 16 * it + 4 * lg);
            const Frag<T, P> Wf[2] = {make_frag<T, P>(E[0], E[1]), make_frag<T, P>(E[2], E[3])};
            const float last = __builtin_amdgcn_exp2f(s.tab()[4 * 64 + 63]);
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                S[i] *= last;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) S[i] = mma(S[i], Sw::cols(s.k(), i, ks, lg, l16), Wf[ks]);
            }
        }
        if (Op::kSets == 1 && c + 1 < nc) __syncthreads();
    }
    if (a.sT && own) {
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(a.sT + so + 16 * i) = S[i];
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads) gdr_reverse_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes;
    constexpr int KT = K / 16, KS = K / 32;
    using Op = Operands<T, K, P>;
    using Sw = Swizzled<T, K>;
    __shared__ __align__(16) char buf[Op::kSets * Op::kBytes];
    const int lane = threadIdx.x & 63, lg = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), slabs = (blockDim.x >> 6) - 1;
    const int64_t seq = blockIdx.z, hv = blockIdx.y, hk = hv / a.group;
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;
    if (wave == slabs) {
        copy_loop<T, K, P, true>(a, buf, lo, hi, slot0, hv, hk, nc - 1, -1, nc, lane);
        return;
    }
    const int64_t col = 16 * ((int64_t)blockIdx.x * slabs + wave) + l16;
    const bool own = 16 * ((int64_t)blockIdx.x * slabs + wave) < a.V;

    f32x4 D[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        D[i] = a.dsT && own ? *reinterpret_cast<const f32x4 *>(a.dsT + so + 16 * i) : zero4();

    T yn[16];
    auto fetch = [&](int64_t c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Cols<T> y(a.dy + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
        for (int i = 0; i < 16; ++i) yn[i] = y.load(i);
    };
    if (own && nc > 0) fetch(nc - 1);
    for (int64_t i = 0; i < nc; ++i) {
        const int64_t c = nc - 1 - i;
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Op s{buf + (Op::kSets == 2 ? (i & 1) * Op::kBytes : 0)};
        __syncthreads();
        if (own) {
            f32x4 dY[4];
#pragma unroll
            for (int j = 0; j < 16; ++j) dY[j >> 2][j & 3] = to_f32(yn[j]);
            if (c > 0) fetch(c - 1);
            const Tiles st(a.st + at.ch * K * a.V, K, a.V, col, lg);
#pragma unroll
            for (int j = 0; j < KT; ++j) st.store(j, D[j]);
            f32x4 dE[4];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) dE[jt] = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const Frag<T, P> Df = make_frag<T, P>(D[2 * ks], D[2 * ks + 1]);
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) dE[jt] = mma(dE[jt], Sw::rows(s.k(), jt, ks, lg, l16), Df);
            }
            {
                const Frag<T, 1> dYf[2] = {make_frag<T, 1>(dY[0], dY[1]), make_frag<T, 1>(dY[2], dY[3])};
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) {
                    dE[jt] *= row4(s.tab(), 2, 16 * jt + 4 * lg);
#pragma unroll
                    for (int ks = jt / 2; ks < 2; ++ks)
                        dE[jt] = mma(dE[jt], load_packed<T, P>(s.p(), up_frag(jt, ks), lane), dYf[ks]);
                }
            }
            f32x4 dR[4];
            {
                const Frag<T, P> dEf[2] = {make_frag<T, P>(dE[0], dE[1]), make_frag<T, P>(dE[2], dE[3])};
                const Tiles rows(a.rows + at.ch * 64 * a.V, 64, a.V, col, lg);
                const Cols<T> dv(a.dv + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) {
                    dR[jt] = zero4();
#pragma unroll
                    for (int ks = jt / 2; ks < 2; ++ks)
                        dR[jt] = mma(dR[jt], load_packed<T, P>(s.t(), up_frag(jt, ks), lane), dEf[ks]);
                    rows.store(jt, dR[jt]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) dv.store(4 * jt + r, dR[jt][r]);
                }
            }
            const float last = __builtin_amdgcn_exp2f(s.tab()[4 * 64 + 63]);
#pragma unroll
            for (int j = 0; j < KT; ++j) D[j] *= last;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                dY[jt] *= row4(s.tab(), 1, 16 * jt + 4 * lg);
                dR[jt] *= -row4(s.tab(), 0, 16 * jt + 4 * lg);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Frag<T, P> Yf = make_frag<T, P>(dY[2 * ks], dY[2 * ks + 1]);
                const Frag<T, P> Rf = make_frag<T, P>(dR[2 * ks], dR[2 * ks + 1]);
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    D[j] = mma(D[j], Sw::cols(s.q(), j, ks, lg, l16), Yf);
                    D[j] = mma(D[j], Sw::cols(s.k(), j, ks, lg, l16), Rf);
                }
            }
        }
        if (Op::kSets == 1 && c > 0) __syncthreads();
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

// Slabs per workgroup, a wave each: as many as there are (8 at most), fewer
// while that leaves compute units without a workgroup.
void scan_grid(const Launch &a, dim3 *grid, dim3 *block)
{
    const int64_t slabs = a.V / 16, units = a.map.nseq * a.Hv;
    int64_t groups = (slabs + 7) / 8;
    while (units * groups < 256 && groups < slabs) ++groups;
    const int64_t per = (slabs + groups - 1) / groups;
    *grid = dim3((unsigned)((slabs + per - 1) / per), (unsigned)a.Hv, (unsigned)a.map.nseq);
    *block = dim3((unsigned)(64 * (per + 1)));   // and the copies'
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
