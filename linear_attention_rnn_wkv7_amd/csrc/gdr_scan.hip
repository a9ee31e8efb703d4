// The scans over the chunks, forward and reverse (the mathematics and the
// operand layouts: gdr_device.h, gdr_factor.h).
//
// One wave owns 16 value columns of one sequence's head: its K x 16 slab of
// the state stays in registers as result tiles, and every product of the
// chain takes its other operand from LDS, so that a chunk needs no exchange
// between waves.  The waves of a workgroup share that operand: K and Q, by
// rows and, through transposing reads, by columns, and the chunk's triangular
// factors.  Those come from memory, or (scan_makes_factors) are made ahead of
// the slabs by waves of their own in the same workgroup and never leave LDS.
//
// Reverse, from the gradient D of the state behind the chunk:
//     dE = P^T dY + w * (K D),  w_j = (gamma_C / gamma_j) beta_j
//     dR = T^T dE  (= dV)
//     D0 = gamma_C D + (gamma Q)^T dY - (gamma K)^T dR
// It leaves D (per chunk) and dR for gdr_grads.hip.
//
// Few, long rows run in segments.  A chunk takes its state on linearly, S1 =
// M S0 + L; a first pass runs every segment from a zero state, and beside it
// K columns that start as the identity and see no values, which gives the
// segment's L and M; a small kernel runs through the segments of a row; the
// second pass starts each from its own state.  (Reverse the same way.)  At 1 x
// 65536 x 32, K = V = 64, bf16, in 8 segments: 0.35 and 0.46 ms for the passes,
// 0.03 between and 0.29 for the factors, 1.12 ms in all; in one piece (as packed
// sequences run) 2.54 ms after the factors.
//
// What bounds them.  fp32: the fp32 matrix instruction (8 x 4096 x 32, K = V =
// 64: 39 GFLOP in 0.34 ms, 112 TFLOP/s of 157; the matrix units are busy 0.7 of
// the time).  bf16: the chain of one chunk, 750 vector and 170 other instructions
// of one wave at K = 64 and one such wave per SIMD (8 x 4096 x 32, with the record:
// 0.30 and 0.32 ms, 64 steps of about 5 us, matrix units busy 0.25 to 0.28); at K =
// 128 1040 and 270, on half of the SIMDs where there are 64 heads (4 x 4096 x 16:
// 0.30 and 0.29 ms, busy 0.15).

#include "gdr_factor.h"

namespace wkv7 {
namespace gdr {
namespace {

// Workgroup n runs on die n % 8: `share` neighbours in order (slab groups, then
// value heads, then sequences) follow one another on one die.
struct Place {
    uint32_t groups, share, total;
    __device__ __forceinline__ uint32_t at(uint32_t n) const
    {
        const uint32_t i = n >> 3;
        return (i / share * 8 + (n & 7)) * share + i % share;   // total or more: none
    }
};

template <typename T>
struct ScanArgs {
    Map map;
    const T *q, *k, *v, *dy;
    const float *s0, *dsT;
    T *y, *dv;
    float *sT, *ds0, *seg_map;
    float *st, *rows;    // record: states and E; reverse: D and dR
    float *table;        // reverse
    const float *g, *beta;
    const char *factors;
    int64_t Hk, Hv, V;
    int group, norm;
    float scale;
    Place place;
};

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
    // The bits, one register to a value: as 16-bit values the compiler would
    // pack them in pairs, and wait for the loads to do so.
    __device__ __forceinline__ uint32_t load(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return __builtin_amdgcn_raw_buffer_load_b32(buf, (int)off(i), 0, 0);
        else
            return __builtin_amdgcn_raw_buffer_load_b16(buf, (int)off(i), 0, 0);
    }
    __device__ static __forceinline__ float value(uint32_t u)
    {
        return sizeof(T) == 4 ? __builtin_bit_cast(float, u) : bf16_lo(u);
    }
    __device__ __forceinline__ void store(int i, float x) const
    {
        if constexpr (sizeof(T) == 4)
            bstore(buf, off(i), x);
        else
            __builtin_amdgcn_raw_buffer_store_b16((unsigned short)pack_bf16(x, x), buf, (int)off(i), 0, 0);
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

// A workgroup's LDS.  kMake: two sets of K and Q, so that the next chunk's
// copies run while one is computed, two of factors, one read and one being
// written, and the scratch of the waves that write them.  Else: two sets of
// all, or one where two do not fit (fp32 with K = 128).
template <typename T, int K>
struct ScanLds {
    static constexpr int kMat = Swizzled<T, K>::kBytes;
    static constexpr int kSets = 2 * (2 * kMat + (int)sizeof(Factor<T>)) <= 160 * 1024 ? 2 : 1;
    char k[kSets][kMat], q[kSets][kMat];
    Factor<T> f[kSets];
};
template <typename T, int K>
struct MakeLds : ScanLds<T, K> {
    FactorLds scratch[kMakers];
};

// The slab into a [V][K] matrix: four rows of a tile are 16 bytes of it.  (By
// single values, [K][V], the 32 stores of K = 128 took 2700 of a step's 11000
// cycles.)
template <int KT>
__device__ __forceinline__ void record_state(float *to, const f32x4 (&S)[KT], int64_t col, int lg)
{
    const uint32_t o = fresh((uint32_t)col * (16 * KT) + 4 * lg);
#pragma unroll
    for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(to + o + 16 * i) = S[i];
}

// When a slab loads its next chunk's values: after the products of the state,
// when the step's operand copies are through, but in the reverse scan with K =
// 128 at the step's start, ahead of the stores of the state.  (At the start
// against after: forward, 1 x 65536 x 32, bf16, second pass 468 and 455 us; 8 x
// 4096 x 32 323 and 306; K = 128, 4 x 4096 x 16, 314 and 300.  Reverse: 8 x 4096 x
// 32 321 and 319; K = 128, 4 x 4096 x 16, 291 and 306.)
template <int K>
constexpr bool kFetchFirst = K == 128;

// The waves of a workgroup run in steps, one chunk of the slabs to a step,
// with a barrier between two steps: the slabs take chunk c in step c (the c-th
// chunk of their direction), its operands arrive in step c - 1.

// One wave copies them from memory (kAll: with Q and P): issuing copies stalls whenever the memory
// system has no room for more, and would stall the products with it.
template <typename T, int K, bool kTrans, bool kAll>
__device__ __forceinline__ void copy_loop(const ScanArgs<T> &a, ScanLds<T, K> &s, int64_t lo, int64_t hi, int64_t slot0,
                                          int64_t hv, int64_t hk, int64_t nc, int lane)
{
    using L = ScanLds<T, K>;
    using F = Factor<T>;
    __builtin_amdgcn_s_setprio(2);
    for (int64_t i = 0; i < nc; ++i) {
        const Pos at = chunk_at(lo, hi, slot0, kTrans ? nc - 1 - i : i, a.Hv, hv);
        const int64_t o = (at.tok * a.Hk + hk) * K;
        const int set = L::kSets == 2 ? (int)(i & 1) : 0;
        if (L::kSets == 1 && i > 0) __syncthreads();   // the only set is free
        dma_rows<T, K>(s.k[set], a.k + o, a.Hk * K, at.len, lane);
        const F *f = reinterpret_cast<const F *>(a.factors) + at.ch;
        if constexpr (kAll) {
            dma_flat<sizeof(F)>(&s.f[set], f, lane);
            dma_rows<T, K>(s.q[set], a.q + o, a.Hk * K, at.len, lane);
        } else {
            dma_flat<sizeof(F::t)>(s.f[set].t, f->t, lane);
            dma_flat<sizeof(F::w)>(s.f[set].w, f->w, lane);
        }
        wait_dma();
        __syncthreads();
    }
}

// kMakers waves take turns at the factors: wave c % kMakers makes those of
// chunk c in steps c - kMakers to c - 1, a stage to a step, and writes them in
// the last.  The wave in its first stage, which waits for memory in any case,
// also copies K and Q for the next step.
template <typename T, int K, bool kTrans>
__device__ __forceinline__ void make_loop(const ScanArgs<T> &a, MakeLds<T, K> &s, int maker, bool tables, int64_t lo,
                                          int64_t hi, int64_t slot0, int64_t hv, int64_t hk, int64_t nc, int lane)
{
    static_assert(MakeLds<T, K>::kSets == 2, "two sets");
    int64_t steps = nc + kMakers - 1;   // barriers still to come
    auto next = [&]() {
        if (steps > 0) __syncthreads();
        --steps;
    };
    for (int i = 0; i < maker; ++i) next();
    for (int64_t i = maker;; i += kMakers) {
        if (steps <= 0) break;
        const int64_t j = i - kMakers + 1;   // the next step's chunk
        const bool made = i < nc;
        const Pos at = chunk_at(lo, hi, slot0, kTrans ? nc - 1 - i : i, a.Hv, hv);
        if (j >= 0 && j < nc) {
            const Pos to = chunk_at(lo, hi, slot0, kTrans ? nc - 1 - j : j, a.Hv, hv);
            const int64_t o = (to.tok * a.Hk + hk) * K;
            dma_rows<T, K>(s.k[j & 1], a.k + o, a.Hk * K, to.len, lane);
            dma_rows<T, K>(s.q[j & 1], a.q + o, a.Hk * K, to.len, lane);
        }
        Factors<T, K, kTrans> f;
        if (made) {
            const int64_t o = (at.tok * a.Hk + hk) * K, og = at.tok * a.Hv + hv;
            f.products(s.scratch[maker], a.k + o, a.q + o, a.g + og, a.beta + og, a.Hk, a.Hv, at.len, a.norm, a.scale,
                       (int)fresh(lane));
        }
        wait_dma();
        next();
        if (made)
            f.decays(s.scratch[maker], kTrans && tables ? a.table + at.ch * kTableFloats : nullptr, at.len, (int)fresh(lane));
        next();
        if (made) f.solve(s.scratch[maker], (int)fresh(lane));
        next();
        Factor<T> &to = s.f[i & 1];
        if (made) f.finish(to.t, to.p, to.w, (int)fresh(lane));
        next();
    }
}

// The waves besides the slabs': returns false in a slab's wave.
template <typename T, int K, bool kTrans, bool kMake, bool kAll>
__device__ __forceinline__ bool feed(const ScanArgs<T> &a, char *buf, int wave, int slabs, bool tables, int64_t lo,
                                     int64_t hi, int64_t slot0, int64_t hv, int64_t hk, int64_t nc, int lane)
{
    if constexpr (kMake) {
        if (wave >= slabs) {
            if (nc > 0)
                make_loop<T, K, kTrans>(a, *reinterpret_cast<MakeLds<T, K> *>(buf), wave - slabs, tables, lo, hi,
                                            slot0, hv, hk, nc, lane);
            return true;
        }
    } else {
        if (wave == slabs) {
            copy_loop<T, K, kTrans, kAll>(a, *reinterpret_cast<ScanLds<T, K> *>(buf), lo, hi, slot0, hv, hk, nc, lane);
            return true;
        }
    }
    return false;
}

// Before a slab's first step.
template <bool kMake>
__device__ __forceinline__ void first_step()
{
    for (int i = 0; i < (kMake ? kMakers : 1); ++i) __syncthreads();
}

// Between two steps of a slab.
template <int kSets>
__device__ __forceinline__ void step_end()
{
    if (kSets == 1) __syncthreads();   // the only set is free: the next copies follow
    __syncthreads();
}

template <typename T, int K, bool kMake>
constexpr int kScanLds = kMake ? (int)sizeof(MakeLds<T, K>) : (int)sizeof(ScanLds<T, K>);
// The most waves: 8 slabs and the copies, or 4 slabs and the makers.
template <bool kMake>
constexpr int kMaxThreads = 64 * (kMake ? 4 + kMakers : 8 + 1);

// kMap: the first pass over segments.
template <typename T, int K, bool kMake, bool kY, bool kMap>
__global__ void __launch_bounds__(kMaxThreads<kMake>) gdr_scan_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes;
    constexpr int KT = K / 16, KS = K / 32;
    using L = ScanLds<T, K>;
    using Sw = Swizzled<T, K>;
    __shared__ __align__(16) char buf[kScanLds<T, K, kMake>];
    L &s = *reinterpret_cast<L *>(buf);
    const int lane = threadIdx.x & 63, lg = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int slabs = (int)(blockDim.x >> 6) - (kMake ? kMakers : 1);
    const uint32_t at = a.place.at(blockIdx.x);
    if (at >= a.place.total) return;
    const uint32_t unit = at / a.place.groups, part = at - unit * a.place.groups;
    const int64_t seq = unit / (uint32_t)a.Hv, hv = unit - (uint32_t)seq * (uint32_t)a.Hv, hk = hv / a.group;
    const int64_t row = seq / a.map.nseg, seg = seq % a.map.nseg, Vc = kMap ? a.V + K : a.V;   // columns
    if (kMap && seg == a.map.nseg - 1) return;   // nothing follows it
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;
    if (feed<T, K, false, kMake, kY>(a, buf, wave, slabs, false, lo, hi, slot0, hv, hk, nc, lane)) return;
    const int64_t col = 16 * ((int64_t)part * slabs + wave) + l16;
    const bool own = 16 * ((int64_t)part * slabs + wave) < Vc;
    const bool extra = kMap && 16 * ((int64_t)part * slabs + wave) >= a.V;   // of the identity

    f32x4 S[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        S[i] = !kMap && a.s0 && own ? *reinterpret_cast<const f32x4 *>(a.s0 + so + 16 * i) : zero4();
    if (extra) {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = 16 * i + 4 * lg + r == col - a.V ? 1.f : 0.f;
    }

    uint32_t vn[16];
    auto fetch = [&](int64_t c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Cols<T> v(a.v + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
        for (int i = 0; i < 16; ++i) vn[i] = extra ? 0u : v.load(i);
    };
    if (own && nc > 0) fetch(0);
    if (nc > 0) first_step<kMake>();
    for (int64_t c = 0; c < nc; ++c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const int set = L::kSets == 2 ? (int)(c & 1) : 0;
        const Factor<T> &f = s.f[set];
        if (own) {
            f32x4 R[4], Y[4];
#pragma unroll
            for (int i = 0; i < 16; ++i) R[i >> 2][i & 3] = Cols<T>::value(vn[i]);
            if (!kMap && a.st) {
                record_state<KT>(a.st + at.ch * K * a.V, S, col, lg);
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
                        acc[it] = mma(acc[it], Sw::rows(s.k[set], it, ks, lg, l16), Sf);
                        if constexpr (kY) Y[it] = mma(Y[it], Sw::rows(s.q[set], it, ks, lg, l16), Sf);
                    }
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) R[it] -= row4(f.w, 0, 16 * it + 4 * lg) * acc[it];
            }
            const Frag<T, P> Rf[2] = {make_frag<T, P>(R[0], R[1]), make_frag<T, P>(R[2], R[3])};
            f32x4 E[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                E[it] = zero4();
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks)
                    E[it] = mma(E[it], load_tri<T, P, false>(f.t, it, ks, lane), Rf[ks]);
            }
            if (c + 1 < nc) fetch(c + 1);
            if (!kMap && a.rows) {
                const Tiles rows(a.rows + at.ch * 64 * a.V, 64, a.V, col, lg);
#pragma unroll
                for (int i = 0; i < 4; ++i) rows.store(i, E[i]);
            }
            if constexpr (kY) {
                const Frag<T, P> Ef[2] = {make_frag<T, P>(E[0], E[1]), make_frag<T, P>(E[2], E[3])};
                const Cols<T> y(a.y + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    Y[it] *= row4(f.w, 1, 16 * it + 4 * lg);
#pragma unroll
                    for (int ks = 0; ks <= it / 2; ++ks)
                        Y[it] = mma(Y[it], load_tri<T, P, false>(f.p, it, ks, lane), Ef[ks]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y.store(4 * it + r, Y[it][r]);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) E[it] *= row4(f.w, 2, 16 * it + 4 * lg);
            const Frag<T, P> Wf[2] = {make_frag<T, P>(E[0], E[1]), make_frag<T, P>(E[2], E[3])};
            const float last = f.w[192];
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                S[i] *= last;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) S[i] = mma(S[i], Sw::cols(s.k[set], i, ks, lg, l16), Wf[ks]);
            }
        }
        if (c + 1 < nc) step_end<L::kSets>();
    }
    if constexpr (kMap) {
        const Tiles out(a.seg_map + (seq * a.Hv + hv) * K * Vc, K, Vc, col, lg);
        if (own) {
#pragma unroll
            for (int i = 0; i < KT; ++i) out.store(i, S[i]);
        }
    } else if (a.sT && own && seg == a.map.nseg - 1) {
        float *to = a.sT + ((row * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(to + 16 * i) = S[i];
    }
}

template <typename T, int K, bool kMake, bool kMap>
__global__ void __launch_bounds__(kMaxThreads<kMake>) gdr_reverse_kernel(ScanArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes;
    constexpr int KT = K / 16, KS = K / 32;
    using L = ScanLds<T, K>;
    using Sw = Swizzled<T, K>;
    __shared__ __align__(16) char buf[kScanLds<T, K, kMake>];
    L &s = *reinterpret_cast<L *>(buf);
    const int lane = threadIdx.x & 63, lg = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int slabs = (int)(blockDim.x >> 6) - (kMake ? kMakers : 1);
    const uint32_t at = a.place.at(blockIdx.x);
    if (at >= a.place.total) return;
    const uint32_t unit = at / a.place.groups, part = at - unit * a.place.groups;
    const int64_t seq = unit / (uint32_t)a.Hv, hv = unit - (uint32_t)seq * (uint32_t)a.Hv, hk = hv / a.group;
    const int64_t row = seq / a.map.nseg, seg = seq % a.map.nseg, Vc = kMap ? a.V + K : a.V;   // columns
    if (kMap && seg == 0) return;   // nothing follows it
    int64_t lo, hi;
    seq_range(a.map, seq, lo, hi);
    const int64_t slot0 = first_slot(a.map, seq, lo), nc = (hi - lo + kChunk - 1) / kChunk;
    if (feed<T, K, true, kMake, true>(a, buf, wave, slabs, part == 0, lo, hi, slot0, hv, hk, nc, lane)) return;
    const int64_t col = 16 * ((int64_t)part * slabs + wave) + l16;
    const bool own = 16 * ((int64_t)part * slabs + wave) < Vc;
    const bool extra = kMap && 16 * ((int64_t)part * slabs + wave) >= a.V;   // of the identity

    f32x4 D[KT];
    const int64_t so = ((seq * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
    for (int i = 0; i < KT; ++i)
        D[i] = !kMap && a.dsT && own ? *reinterpret_cast<const f32x4 *>(a.dsT + so + 16 * i) : zero4();
    if (extra) {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) D[i][r] = 16 * i + 4 * lg + r == col - a.V ? 1.f : 0.f;
    }

    uint32_t yn[16];
    auto fetch = [&](int64_t c) {
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const Cols<T> y(a.dy + (at.tok * a.Hv + hv) * a.V, a.Hv * a.V, a.V, col, at.len, lg);
#pragma unroll
        for (int i = 0; i < 16; ++i) yn[i] = extra ? 0u : y.load(i);
    };
    if (own && nc > 0) fetch(nc - 1);
    if (nc > 0) first_step<kMake>();
    for (int64_t i = 0; i < nc; ++i) {
        const int64_t c = nc - 1 - i;
        const Pos at = chunk_at(lo, hi, slot0, c, a.Hv, hv);
        const int set = L::kSets == 2 ? (int)(i & 1) : 0;
        const Factor<T> &f = s.f[set];
        if (own) {
            f32x4 dY[4];
#pragma unroll
            for (int j = 0; j < 16; ++j) dY[j >> 2][j & 3] = Cols<T>::value(yn[j]);
            if (kFetchFirst<K> && c > 0) fetch(c - 1);
            if constexpr (!kMap) {
                record_state<KT>(a.st + at.ch * K * a.V, D, col, lg);
            }
            f32x4 dE[4];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) dE[jt] = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const Frag<T, P> Df = make_frag<T, P>(D[2 * ks], D[2 * ks + 1]);
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) dE[jt] = mma(dE[jt], Sw::rows(s.k[set], jt, ks, lg, l16), Df);
            }
            {
                const Frag<T, 1> dYf[2] = {make_frag<T, 1>(dY[0], dY[1]), make_frag<T, 1>(dY[2], dY[3])};
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) {
                    dE[jt] *= row4(f.w, 2, 16 * jt + 4 * lg);
#pragma unroll
                    for (int ks = jt / 2; ks < 2; ++ks)
                        dE[jt] = mma(dE[jt], load_tri<T, P, true>(f.p, jt, ks, lane), dYf[ks]);
                }
            }
            if (!kFetchFirst<K> && c > 0) fetch(c - 1);
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
                        dR[jt] = mma(dR[jt], load_tri<T, P, true>(f.t, jt, ks, lane), dEf[ks]);
                    if constexpr (!kMap) {
                        rows.store(jt, dR[jt]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) dv.store(4 * jt + r, dR[jt][r]);
                    }
                }
            }
            const float last = f.w[192];
#pragma unroll
            for (int j = 0; j < KT; ++j) D[j] *= last;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                dY[jt] *= row4(f.w, 1, 16 * jt + 4 * lg);
                dR[jt] *= -row4(f.w, 0, 16 * jt + 4 * lg);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Frag<T, P> Yf = make_frag<T, P>(dY[2 * ks], dY[2 * ks + 1]);
                const Frag<T, P> Rf = make_frag<T, P>(dR[2 * ks], dR[2 * ks + 1]);
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    D[j] = mma(D[j], Sw::cols(s.q[set], j, ks, lg, l16), Yf);
                    D[j] = mma(D[j], Sw::cols(s.k[set], j, ks, lg, l16), Rf);
                }
            }
        }
        if (c > 0) step_end<L::kSets>();
    }
    if constexpr (kMap) {
        const Tiles out(a.seg_map + (seq * a.Hv + hv) * K * Vc, K, Vc, col, lg);
        if (own) {
#pragma unroll
            for (int i = 0; i < KT; ++i) out.store(i, D[i]);
        }
    } else if (a.ds0 && own && seg == 0) {
        float *to = a.ds0 + ((row * a.Hv + hv) * a.V + col) * K + 4 * lg;
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(to + 16 * i) = D[i];
    }
}

// The states the segments of a row start from: S behind a segment is L + M S,
// of the state before it.  One wave per 16 columns of a row's head; kReverse:
// from the last segment to the first.
template <int K, bool kReverse>
__global__ void __launch_bounds__(64) gdr_carry_kernel(const float *from, const float *seg_map, float *carry, int nseg,
                                                       int64_t Hv, int64_t V)
{
    constexpr int KT = K / 16;
    const int lane = threadIdx.x, lg = lane >> 4, l16 = lane & 15;
    const int64_t row = blockIdx.z, hv = blockIdx.y, col = 16 * (int64_t)blockIdx.x + l16, Vc = V + K;
    f32x4 S[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
        S[i] = from ? *reinterpret_cast<const f32x4 *>(from + ((row * Hv + hv) * V + col) * K + 16 * i + 4 * lg) : zero4();
    for (int n = 0; n < nseg; ++n) {
        const int64_t seq = row * nseg + (kReverse ? nseg - 1 - n : n);
        float *to = carry + ((seq * Hv + hv) * V + col) * K + 4 * lg;
#pragma unroll
        for (int i = 0; i < KT; ++i) *reinterpret_cast<f32x4 *>(to + 16 * i) = S[i];
        if (n + 1 == nseg) break;
        const float *m = seg_map + (seq * Hv + hv) * K * Vc;
        f32x4 N[KT];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) N[i][r] = m[(16 * i + 4 * lg + r) * Vc + col];
#pragma unroll
            for (int k = 0; k < KT; ++k)
                N[i] = mma16(N[i], *reinterpret_cast<const f32x4 *>(m + (16 * i + l16) * Vc + V + 16 * k + 4 * lg), S[k]);
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) S[i] = N[i];
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
    p.g = a.g;
    p.beta = a.beta;
    p.norm = a.norm;
    p.scale = a.scale;
    p.factors = static_cast<const char *>(a.factors);
    p.seg_map = a.seg_map;
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.V = a.V;
    p.group = (int)(a.Hv / a.Hk);
    return p;
}

Place place_of(const ScanGrid &g) { return Place{(uint32_t)g.groups, (uint32_t)g.share, (uint32_t)g.total}; }

template <typename T, int K, bool kMake>
hipError_t scan_t(const Launch &a, bool reverse, hipStream_t stream)
{
    ScanArgs<T> p = scan_args<T>(a);
    const int64_t units = a.map.nseq * a.map.nseg * a.Hv;
    if constexpr (!kMake) {
        if (a.map.nseg > 1) {
            const ScanGrid g = scan_grid(units, p.group, a.V + K, false);
            const dim3 grid((unsigned)g.blocks), block((unsigned)g.threads);
            p.place = place_of(g);
            const dim3 rows((unsigned)(a.V / 16), (unsigned)a.Hv, (unsigned)a.map.nseq);
            if (reverse) {
                hipLaunchKernelGGL((gdr_reverse_kernel<T, K, false, true>), grid, block, 0, stream, p);
                hipLaunchKernelGGL((gdr_carry_kernel<K, true>), rows, dim3(64), 0, stream, a.dsT, a.seg_map, a.carry,
                                   (int)a.map.nseg, a.Hv, a.V);
                p.dsT = a.carry;
            } else {
                hipLaunchKernelGGL((gdr_scan_kernel<T, K, false, false, true>), grid, block, 0, stream, p);
                hipLaunchKernelGGL((gdr_carry_kernel<K, false>), rows, dim3(64), 0, stream, a.s0, a.seg_map, a.carry,
                                   (int)a.map.nseg, a.Hv, a.V);
                p.s0 = a.carry;
            }
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    const ScanGrid g = scan_grid(units, p.group, a.V, kMake);
    const dim3 grid((unsigned)g.blocks), block((unsigned)g.threads);
    p.place = place_of(g);
    if (reverse) {
        p.st = a.ws_ds;
        p.rows = a.ws_dr;
        hipLaunchKernelGGL((gdr_reverse_kernel<T, K, kMake, false>), grid, block, 0, stream, p);
    } else if (a.y) {
        hipLaunchKernelGGL((gdr_scan_kernel<T, K, kMake, true, false>), grid, block, 0, stream, p);
    } else {
        hipLaunchKernelGGL((gdr_scan_kernel<T, K, kMake, false, false>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

hipError_t scan_any(const Launch &a, bool reverse, hipStream_t stream)
{
    if (!a.factors) return scan_t<bf16, 64, true>(a, reverse, stream);
    const hipError_t e = launch_prep(a, reverse, stream);
    if (e != hipSuccess) return e;
    if (a.dtype == WKV7_F32)
        return a.K == 64 ? scan_t<float, 64, false>(a, reverse, stream) : scan_t<float, 128, false>(a, reverse, stream);
    return a.K == 64 ? scan_t<bf16, 64, false>(a, reverse, stream) : scan_t<bf16, 128, false>(a, reverse, stream);
}

}  // namespace

hipError_t launch_scan(const Launch &a, hipStream_t stream) { return scan_any(a, false, stream); }
hipError_t launch_reverse(const Launch &a, hipStream_t stream) { return scan_any(a, true, stream); }

}  // namespace gdr
}  // namespace wkv7
