// The triangular factors of a chunk of the gated delta rule, by one wave:
//     T = (I + N diag(beta))^-1,  N_ij = Gamma_ij k_i . k_j     (i > j)
//     P_ij = beta_j Gamma_ij q_i . k_j                          (i >= j)
// and the chunk's row weights.  q . k and k . k run on the matrix cores
// straight from memory; the decays, and under GDR_NORM_QK the reciprocal
// lengths rk, rq of k and q, are applied to the products, so that q and k
// enter as they are.
//
// T is formed by forward substitution inside its four diagonal 16 x 16
// blocks (one lane per block and column), X_jj, and from those by blocks on
// fp32 matrix instructions, with L = N diag(beta).  A tile in D layout is the
// left operand of its transpose, so whichever of T and T^T is wanted as a left
// operand is formed from the other's tiles:
//     (I + L) T = I:  X_ij = -X_ii sum_{k = j}^{i-1} L_ik X_kj         (T^T)
//     T (I + L) = I:  X_ij^T = -X_jj^T sum_{k = j+1}^{i} L_kj^T X_ik^T  (T)
// (Powers of L would need fewer dependent steps, but for keys that are alike
// they grow like binomials and cancel.)
//
// Tokens behind the sequence's end count as k = q = 0, g = 0, beta = 0.
#pragma once

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {

// A triangle's ten 16 x 16 tiles, row by row.
__device__ __forceinline__ constexpr int tile_id(int i, int j) { return i * (i + 1) / 2 + j; }

// As operands (kTri elements per part): for a tile, each lane's four values,
// row l16 and columns 4 lg .. 4 lg + 3 of the tile or, kTrans, of its
// transpose.  In bf16, tiles that make up one 32-deep step of an operand lie
// side by side in a lane's 16 bytes; the two that stand alone in theirs share
// the last place.
constexpr int kTri = 10 * 64 * 4;
template <bool kTrans>
__device__ __forceinline__ constexpr int tri_place(int tile)
{
    return (int)((kTrans ? 0x9753642810ull : 0x7654932108ull) >> (4 * tile)) & 15;
}
template <typename T, bool kTrans>
__device__ __forceinline__ constexpr int tri_at(int tile, int lane)
{
    if (sizeof(T) == 4) return (tile * 64 + lane) * 4;
    return ((tri_place<kTrans>(tile) >> 1) * 64 + lane) * 8 + (tri_place<kTrans>(tile) & 1) * 4;
}

// Row tile `it` of a lower triangle (steps 0 .. it / 2), or of a transposed
// one (steps it / 2 .. 1), as the left operand of step ks.
template <typename T, int P, bool kTrans>
__device__ __forceinline__ Frag<T, P> load_tri(const T *base, int it, int ks, int lane)
{
    using Quad = typename Num<T>::Quad;
    Frag<T, P> f;
    const bool lo = kTrans ? 2 * ks >= it : true, hi = kTrans ? true : 2 * ks + 1 <= it;   // tiles of the triangle
    const int a = kTrans ? tile_id(2 * ks, it) : tile_id(it, 2 * ks), b = kTrans ? tile_id(2 * ks + 1, it) : tile_id(it, 2 * ks + 1);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (lo && hi && sizeof(T) == 4) {
            f.p[p] = __builtin_shufflevector(*reinterpret_cast<const Quad *>(base + p * kTri + tri_at<T, kTrans>(a, lane)),
                                             *reinterpret_cast<const Quad *>(base + p * kTri + tri_at<T, kTrans>(b, lane)),
                                             0, 1, 2, 3, 4, 5, 6, 7);
        } else if (lo && hi) {
            f.p[p] = *reinterpret_cast<const typename Num<T>::Oct *>(base + p * kTri + tri_at<T, kTrans>(a, lane));
        } else {
            const Quad x = *reinterpret_cast<const Quad *>(base + p * kTri + tri_at<T, kTrans>(lo ? a : b, lane));
            f.p[p] = lo ? __builtin_shufflevector(x, Quad{}, 0, 1, 2, 3, 4, 5, 6, 7)
                        : __builtin_shufflevector(Quad{}, x, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    return f;
}

// A chunk's row weights: gamma_i rk, gamma_i rq scale, (gamma_C / gamma_i) rk
// beta_i, and gamma_C.
constexpr int kWeights = 256;

// A chunk's factors as the scan reads them, T and P in the parts of an fp32
// operand (1 KB copies move it whole).
template <typename T>
struct Factor {
    T t[Num<T>::kPlanes * kTri], p[Num<T>::kPlanes * kTri];
    float w[kWeights];
};

// LDS of one such wave: ten tiles.  Rows r, r + 4, r + 8, r + 12 lie side by
// side, and the 16-byte pieces of a row are permuted, so that neither writes
// of a result tile nor 16-byte reads of 16 rows meet a bank twice.
constexpr int kTile = 256;
__device__ __forceinline__ constexpr int in_tile(int row, int col)
{
    return ((row & 3) * 4 + (row >> 2)) * 16 + (((col >> 2) ^ (row & 3)) << 2 | (col & 3));
}
struct FactorLds {
    float t[10 * kTile];
    float rq[64], rk[64], Gh[64], Gl[64], cb[64];
};

__device__ __forceinline__ f32x4 mma16(f32x4 c, f32x4 a, f32x4 b)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

// Tiles in D layout as left operands of their transposes, in P parts.
template <typename T, int P, bool kTrans>
__device__ __forceinline__ void write_tri(T *out, const f32x4 (&X)[10], int lane)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int t = 0; t < 10; ++t) *reinterpret_cast<f32x4 *>(out + tri_at<T, kTrans>(t, lane)) = X[t];
        return;
    }
#pragma unroll
    for (int i = 0; i < 10; i += 2) {   // places i, i + 1
        f32x4 x[2];
#pragma unroll
        for (int t = 0; t < 10; ++t) {
            if (tri_place<kTrans>(t) == i) x[0] = X[t];
            if (tri_place<kTrans>(t) == i + 1) x[1] = X[t];
        }
        const Frag<T, P> f = make_frag<T, P>(x[0], x[1]);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<typename Num<T>::Oct *>(out + p * kTri + (i / 2 * 64 + lane) * 8) = f.p[p];
    }
}

// Four stages with state between them in registers and the wave's LDS.
template <typename T, int K, bool kTrans>
struct Factors {
    f32x4 kk[10], qk[10];   // K K^T and Q K^T, then L and P, then T and P
    float g, be;            // lane = token
    float wa, wb, we, last;

    // kk, qk, and the rows' lengths
    __device__ __forceinline__ void products(FactorLds &s, const T *k, const T *q, const float *gp, const float *bp,
                                             int64_t Hk, int64_t Hv, int len, bool norm, float scale, int lane)
    {
        using Oct = typename Num<T>::Oct;
        const int lg = lane >> 4, l16 = lane & 15;
        const bool in = lane < len;
        g = in ? gp[lane * Hv] : 0.f;
        be = in ? bp[lane * Hv] : 0.f;
        float nq[4], nk[4];
#pragma unroll
        for (int i = 0; i < 10; ++i) kk[i] = qk[i] = zero4();
#pragma unroll
        for (int i = 0; i < 4; ++i) nq[i] = nk[i] = 0.f;
#pragma unroll 1   // registers
        for (int ks = 0; ks < K / 32; ++ks) {
            Frag<T, 1> fk[4], fq[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                fk[it].p[0] = fq[it].p[0] = Oct{};
                const int t = 16 * it + l16;
                if (t < len) {
                    const uint32_t o = (uint32_t)t * (uint32_t)(Hk * K) + 32 * ks + 8 * lg;
                    fk[it].p[0] = *reinterpret_cast<const Oct *>(k + o);
                    fq[it].p[0] = *reinterpret_cast<const Oct *>(q + o);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
#pragma unroll
                for (int jt = 0; jt <= it; ++jt) {
                    kk[tile_id(it, jt)] = mma(kk[tile_id(it, jt)], fk[it], fk[jt]);
                    qk[tile_id(it, jt)] = mma(qk[tile_id(it, jt)], fq[it], fk[jt]);
                }
                if (norm) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        nq[it] = fmaf(to_f32(fq[it].p[0][j]), to_f32(fq[it].p[0][j]), nq[it]);
                        nk[it] = fmaf(to_f32(fk[it].p[0][j]), to_f32(fk[it].p[0][j]), nk[it]);
                    }
                }
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            float x = scale, z = 1.f;
            if (norm) {
                nq[it] += __shfl_xor(nq[it], 16);
                nk[it] += __shfl_xor(nk[it], 16);
                nq[it] += __shfl_xor(nq[it], 32);
                nk[it] += __shfl_xor(nk[it], 32);
                x = scale / sqrtf(nq[it] + 1e-6f);
                z = 1.f / sqrtf(nk[it] + 1e-6f);
            }
            if (lg == 0) {
                s.rq[16 * it + l16] = x;
                s.rk[16 * it + l16] = z;
            }
        }
        wave_sync();
    }

    // the decays; L and the inverses of its diagonal blocks in LDS, P in qk.
    // table (may be null) receives the rows that gdr_grads.hip uses.
    __device__ __forceinline__ void decays(FactorLds &s, float *table, int len, int lane)
    {
        const int lg = lane >> 4, l16 = lane & 15;
        const bool in = lane < len;
        const float rql = s.rq[lane], rkl = s.rk[lane];
        const float gc = g < -200.f ? -200.f : g;   // exp is zero there; keeps differences finite
        double G = (double)gc * 1.4426950408889634074;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(G, d);
            if (lane >= d) G += up;
        }
        const double end = __shfl(G, 63);
        const float hi = (float)G, lo = (float)(G - (double)hi);
        const float ga = __builtin_amdgcn_exp2f(hi), eh = __builtin_amdgcn_exp2f((float)(end - G));
        s.Gh[lane] = hi;
        s.Gl[lane] = lo;
        s.cb[lane] = be * rkl;
        wa = in ? ga * rkl : 0.f;
        wb = in ? ga * rql : 0.f;
        we = in ? eh * rkl * be : 0.f;
        last = __builtin_amdgcn_exp2f((float)end);
        if (table) {
            table[lane] = hi;
            table[64 + lane] = lo;
            table[128 + lane] = be;
            table[192 + lane] = rkl;
            table[256 + lane] = rql;
        }
        wave_sync();
        float Ghj[4], Glj[4], cj[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            Ghj[jt] = s.Gh[16 * jt + l16];
            Glj[jt] = s.Gl[16 * jt + l16];
            cj[jt] = s.cb[16 * jt + l16];
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i0 = 16 * it + 4 * lg;
            const f32x4 gh = *reinterpret_cast<const f32x4 *>(s.Gh + i0), gl = *reinterpret_cast<const f32x4 *>(s.Gl + i0);
            const f32x4 rk = *reinterpret_cast<const f32x4 *>(s.rk + i0), rq = *reinterpret_cast<const f32x4 *>(s.rq + i0);
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                const int id = tile_id(it, jt);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float gb = __builtin_amdgcn_exp2f((gh[r] - Ghj[jt]) + (gl[r] - Glj[jt])) * cj[jt];
                    const bool low = it > jt || 4 * lg + r > l16, diag = it == jt && 4 * lg + r == l16;
                    kk[id][r] = low ? kk[id][r] * rk[r] * gb : 0.f;
                    qk[id][r] = low || diag ? qk[id][r] * rq[r] * gb : 0.f;
                    // the transposed recurrence takes L as a left operand itself
                    if (it == jt || kTrans) s.t[id * kTile + in_tile(4 * lg + r, l16)] = kk[id][r];
                }
            }
        }
        wave_sync();
        // lane (lg, l16) solves column l16 of diagonal block lg
        float *L = s.t + tile_id(lg, lg) * kTile;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);   // else all of L is read at once
            float acc = r == l16 ? 1.f : 0.f;
#pragma unroll
            for (int q4 = 0; q4 < r; q4 += 4) {
                const f32x4 l = *reinterpret_cast<const f32x4 *>(L + in_tile(r, q4));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q4 + q < r) acc = fmaf(-l[q], x[q4 + q], acc);
            }
            x[r] = acc;
        }
        wave_sync();
#pragma unroll
        for (int r = 0; r < 16; ++r) L[in_tile(r, l16)] = x[r];
        wave_sync();
    }

    // the rest of T, in kk: D layout of T (kTrans) or of T^T
    __device__ __forceinline__ void solve(FactorLds &s, int lane)
    {
        const int lg = lane >> 4, l16 = lane & 15;
        f32x4 X[10], dia[4];   // dia: the diagonal blocks as left operands
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *d = s.t + tile_id(i, i) * kTile;
            const f32x4 row = *reinterpret_cast<const f32x4 *>(d + in_tile(l16, 4 * lg));
            f32x4 col;
#pragma unroll
            for (int r = 0; r < 4; ++r) col[r] = d[in_tile(4 * lg + r, l16)];
            X[tile_id(i, i)] = kTrans ? col : row;
            dia[i] = kTrans ? row : col;
        }
#pragma unroll
        for (int n = 1; n < 4; ++n) {   // block diagonal by block diagonal
#pragma unroll
            for (int j = 0; j + n < 4; ++j) {
                const int i = j + n;
                f32x4 acc = zero4();
                if constexpr (kTrans) {
#pragma unroll
                    for (int k = j; k < i; ++k) {
                        const f32x4 l = *reinterpret_cast<const f32x4 *>(s.t + tile_id(i, k) * kTile + in_tile(l16, 4 * lg));
                        acc = mma16(acc, l, X[tile_id(k, j)]);
                    }
                    X[tile_id(i, j)] = -mma16(zero4(), dia[i], acc);
                } else {
#pragma unroll
                    for (int k = j + 1; k <= i; ++k) acc = mma16(acc, kk[tile_id(k, j)], X[tile_id(i, k)]);
                    X[tile_id(i, j)] = -mma16(zero4(), dia[j], acc);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) kk[i] = X[i];
        if constexpr (!kTrans) {   // P^T in D layout
            wave_sync();
#pragma unroll
            for (int i = 0; i < 10; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s.t[i * kTile + in_tile(4 * lg + r, l16)] = qk[i][r];
            wave_sync();
#pragma unroll
            for (int i = 0; i < 10; ++i) qk[i] = *reinterpret_cast<const f32x4 *>(s.t + i * kTile + in_tile(l16, 4 * lg));
            wave_sync();
        }
    }

    // T and P (kTrans: their transposes) and the weights to where the scan
    // reads them
    __device__ __forceinline__ void finish(T *t, T *p, float *weights, int lane)
    {
        write_tri<T, Num<T>::kPlanes, kTrans>(t, kk, lane);
        write_tri<T, Num<T>::kPlanes, kTrans>(p, qk, lane);
        weights[lane] = wa;
        weights[64 + lane] = wb;
        weights[128 + lane] = we;
        weights[192 + lane] = last;
    }
};

}  // namespace gdr
}  // namespace wkv7
