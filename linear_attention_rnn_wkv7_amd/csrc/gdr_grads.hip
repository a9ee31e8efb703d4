// dq, dk, dg and dbeta of every chunk, from the state S before it, the
// gradient D of the state behind it, and its rows E, dR, dY (gdr_device.h,
// gdr_scan.hip).  With M1 = dY S^T, M2 = dR S^T, M3 = E D^T  [C, K] and
// Z = dY E^T (i >= j), X = dR E^T (i > j)  [C, C], q and k as normalised and
// q scaled:
//     dq_i = gamma_i M1_i + sum_j (beta_j Gamma_ij Z_ij) k_j
//     dk_i = A_i + beta_i F_i
//     A_i  = -gamma_i M2_i - sum_j (beta_j Gamma_ij X_ij) k_j
//     F_j  = e_j M3_j + sum_i Gamma_ij (Z_ij q_i - X_ij k_i),  e = gamma_C / gamma
//     dbeta_j = k_j . F_j
//     dG_i = q_i . dq_i + k_i . A_i - beta_i k_i . F_i   (+ at the chunk's end
//            sum_j beta_j e_j k_j . M3_j + gamma_C <S, D>),
// and dg is the reverse cumulative sum of dG.  (Every term that G_i, beta_i
// enter is a row dot of what dq, dk are made of, so no C x C array besides Z
// and X is needed.)
//
// One workgroup of four waves per chunk and key head; it adds up the group's
// value heads in registers.  Each wave owns K / 4 key columns: it reads its
// rows of S and D once from memory as operands, and shares E, dR, dY in LDS.
// Z and X tiles go through LDS into operand order once per chunk.

#include "gdr_factor.h"

namespace wkv7 {
namespace gdr {
namespace {

template <typename T>
struct GradArgs {
    Map map;
    const T *q, *k, *dy;
    const float *S, *D, *E, *dR, *table;
    T *dq, *dk;
    float *dg, *dbeta;
    int64_t Hk, Hv, V;
    int group, norm;
    float scale;
};

template <typename T, int K>
struct GradLds {
    static constexpr int P = Num<T>::kPlanes, LT = 64 + kPad<T>;
    T kt[K * LT], qt[K * LT];
    union {
        struct {
            T dy[64 * LT], dr[P * 64 * LT], e[P * 64 * LT];
        } in;
        T w[4][P * kTri];   // W1, W2 (for dq, A), then transposed (for F)
    } u;
    float tab[kTableFloats], gam[64], eh[64];
    float red[4][4][64];       // per wave: q.dq, k.A, k.F, k.M3
    float ip[4];               // <S, D>
    float tq[64], tk[64];      // over the group: q.dq, k.dk
};

template <typename T, int P>
__device__ __forceinline__ void put(T *dst, int at, f32x4 x)   // 4 consecutive elements
{
    typename Num<T>::Quad q[P];
    split_quad<T, P>(x, q);
#pragma unroll
    for (int i = 0; i < P; ++i) *reinterpret_cast<typename Num<T>::Quad *>(dst + i * kTri + at) = q[i];
}

template <typename T, int P>
__device__ __forceinline__ void put1(T *dst, int at, float x)
{
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const T z = (T)x;
        dst[i * kTri + at] = z;
        x -= (float)z;
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(256) gdr_grads_kernel(GradArgs<T> a)
{
    using L = GradLds<T, K>;
    using Quad = typename Num<T>::Quad;
    constexpr int P = L::P, LT = L::LT, NT = K / 64;   // 16-column tiles per wave
    __shared__ __align__(16) char buf[sizeof(L)];
    L &s = *reinterpret_cast<L *>(buf);
    const int64_t slot = blockIdx.x, hk = blockIdx.y;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, lg = lane >> 4, l16 = lane & 15;

    for (int b = tid; b < 2 * 16 * (K / 4); b += 256) {
        const int which = b / (16 * (K / 4)), i0 = b % (16 * (K / 4));
        const int col = 4 * (i0 % (K / 4)), t0 = 4 * (i0 / (K / 4));
        const T *src = (which ? a.k : a.q) + ((c.tok + t0) * a.Hk + hk) * K + col;
        T *dst = which ? s.kt : s.qt;
        Quad x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = Quad{};
            if (t0 + r < c.len) x[r] = *reinterpret_cast<const Quad *>(src + r * a.Hk * K);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<Quad *>(dst + (col + i) * LT + kpos(t0)) = Quad{x[0][i], x[1][i], x[2][i], x[3][i]};
    }
    if (tid < 64) s.tq[tid] = s.tk[tid] = 0.f;

    f32x4 dq[4][NT], dk[4][NT];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int n = 0; n < NT; ++n) dq[it][n] = dk[it][n] = zero4();

    for (int gi = 0; gi < a.group; ++gi) {
        const int64_t hv = hk * a.group + gi, ch = slot * a.Hv + hv;
        __syncthreads();
        for (int i = tid; i < kTableFloats / 4; i += 256)
            reinterpret_cast<f32x4 *>(s.tab)[i] = reinterpret_cast<const f32x4 *>(a.table + ch * kTableFloats)[i];
        f32x4 M1[4][NT], M2[4][NT], M3[4][NT], Z[4], X[4];
        float ip = 0.f;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            Z[it] = X[it] = zero4();
#pragma unroll
            for (int n = 0; n < NT; ++n) M1[it][n] = M2[it][n] = M3[it][n] = zero4();
        }
        for (int64_t v0 = 0; v0 < a.V; v0 += 64) {
            __syncthreads();
            for (int b = tid; b < 64 * 16; b += 256) {
                const int t = b >> 4, v = 4 * (b & 15);
                const bool in = v0 + v < a.V;
                Quad x = {};
                f32x4 r = zero4(), e = zero4();
                if (in) {
                    if (t < c.len)
                        x = *reinterpret_cast<const Quad *>(a.dy + ((c.tok + t) * a.Hv + hv) * a.V + v0 + v);
                    r = *reinterpret_cast<const f32x4 *>(a.dR + (ch * 64 + t) * a.V + v0 + v);
                    e = *reinterpret_cast<const f32x4 *>(a.E + (ch * 64 + t) * a.V + v0 + v);
                }
                const int at = t * LT + kpos(v);
                *reinterpret_cast<Quad *>(s.u.in.dy + at) = x;
                Quad rz[P], ez[P];
                split_quad<T, P>(r, rz);
                split_quad<T, P>(e, ez);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    *reinterpret_cast<Quad *>(s.u.in.dr + p * 64 * LT + at) = rz[p];
                    *reinterpret_cast<Quad *>(s.u.in.e + p * 64 * LT + at) = ez[p];
                }
            }
            __syncthreads();
#pragma unroll
            for (int vs = 0; vs < 2; ++vs) {
                Frag<T, P> Sf[NT], Df[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 x[2], d[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[h] = d[h] = zero4();
                        const int64_t v = v0 + 32 * vs + 16 * h + 4 * lg;
                        const int64_t o = (ch * K + 16 * (NT * w + n) + l16) * a.V + v;
                        if (v < a.V) {
                            x[h] = *reinterpret_cast<const f32x4 *>(a.S + o);
                            d[h] = *reinterpret_cast<const f32x4 *>(a.D + o);
                        }
                        const f32x4 xd = x[h] * d[h];
                        ip += (xd[0] + xd[1]) + (xd[2] + xd[3]);
                    }
                    Sf[n] = make_frag<T, P>(x[0], x[1]);
                    Df[n] = make_frag<T, P>(d[0], d[1]);
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const Frag<T, 1> y = load_frag<T, 1>(s.u.in.dy, 16 * it + l16, LT, vs, lg, 0);
                    const Frag<T, P> r = load_frag<T, P>(s.u.in.dr, 16 * it + l16, LT, vs, lg, 64 * LT);
                    const Frag<T, P> e = load_frag<T, P>(s.u.in.e, 16 * it + l16, LT, vs, lg, 64 * LT);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        M1[it][n] = mma(M1[it][n], y, Sf[n]);
                        M2[it][n] = mma(M2[it][n], r, Sf[n]);
                        M3[it][n] = mma(M3[it][n], e, Df[n]);
                    }
                }
                // Z column tile w, X column tile 3 - w: five tiles per wave
                const Frag<T, P> ez = load_frag<T, P>(s.u.in.e, 16 * w + l16, LT, vs, lg, 64 * LT);
                const Frag<T, P> ex = load_frag<T, P>(s.u.in.e, 16 * (3 - w) + l16, LT, vs, lg, 64 * LT);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    if (it >= w)
                        Z[it] = mma(Z[it], load_frag<T, 1>(s.u.in.dy, 16 * it + l16, LT, vs, lg, 0), ez);
                    if (it >= 3 - w)
                        X[it] = mma(X[it], load_frag<T, P>(s.u.in.dr, 16 * it + l16, LT, vs, lg, 64 * LT), ex);
                }
            }
        }
        if (tid < 64) {
            const float G = s.tab[tid] + s.tab[64 + tid];
            const float dhi = s.tab[63] - s.tab[tid], dlo = s.tab[64 + 63] - s.tab[64 + tid];
            s.gam[tid] = __builtin_amdgcn_exp2f(G);
            s.eh[tid] = __builtin_amdgcn_exp2f(dhi + dlo);
        }
        ip = wave_sum(ip);
        if (lane == 0) s.ip[w] = ip;
        __syncthreads();   // E, dR, dY are done with; the table is there
        // Z and X with their decays, as operands
#pragma unroll
        for (int zx = 0; zx < 2; ++zx) {
            const int jt = zx ? 3 - w : w, j = 16 * jt + l16;
            const float Ghj = s.tab[j], Glj = s.tab[64 + j];
            const float cj = s.tab[2 * 64 + j] * s.tab[3 * 64 + j];   // beta rk
            T *wa = s.u.w[zx], *wt = s.u.w[2 + zx];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                if (it < jt) continue;
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * it + 4 * lg + r;
                    float v = 0.f;
                    if (zx ? i > j : i >= j) {
                        const float gd = __builtin_amdgcn_exp2f((s.tab[i] - Ghj) + (s.tab[64 + i] - Glj));
                        v = gd * (zx ? -X[it][r] : Z[it][r]);
                    }
                    // row i, k = j
                    put1<T, P>(wa, (tile_id(it, jt) * 64 + (l16 >> 2) * 16 + 4 * lg + r) * 4 + (l16 & 3), v * cj);
                    x[r] = v * s.tab[(zx ? 3 : 4) * 64 + i];
                }
                // row j, k = i
                put<T, P>(wt, (tile_id(it, jt) * 64 + lane) * 4, x);
            }
        }
        __syncthreads();
        float qd[16], ka[16], kf[16], km[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) qd[i] = ka[i] = kf[i] = km[i] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int kc = 16 * (NT * w + n) + l16;   // this lane's key column
            Frag<T, 1> kf2[2], qf2[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                kf2[ks] = load_frag<T, 1>(s.kt, kc, LT, ks, lg, 0);
                qf2[ks] = load_frag<T, 1>(s.qt, kc, LT, ks, lg, 0);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const f32x4 gam = *reinterpret_cast<const f32x4 *>(s.gam + 16 * it + 4 * lg);
                const f32x4 eh = *reinterpret_cast<const f32x4 *>(s.eh + 16 * it + 4 * lg);
                const f32x4 be = row4(s.tab, 2, 16 * it + 4 * lg);
                const f32x4 rk = row4(s.tab, 3, 16 * it + 4 * lg), rq = row4(s.tab, 4, 16 * it + 4 * lg);
                f32x4 q1 = gam * M1[it][n], A = -gam * M2[it][n], m3 = eh * M3[it][n], F = m3;
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks) {
                    q1 = mma(q1, load_tri<T, P, false>(s.u.w[0], it, ks, lane), kf2[ks]);
                    A = mma(A, load_tri<T, P, false>(s.u.w[1], it, ks, lane), kf2[ks]);
                }
#pragma unroll
                for (int ks = it / 2; ks < 2; ++ks) {
                    F = mma(F, load_tri<T, P, true>(s.u.w[2], it, ks, lane), qf2[ks]);
                    F = mma(F, load_tri<T, P, true>(s.u.w[3], it, ks, lane), kf2[ks]);
                }
                // this lane's q, k of the tile: rows 16 it + 4 lg + r
                f32x4 kv, qv;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    kv[r] = to_f32(kf2[it >> 1].p[0][(it & 1) * 4 + r]);
                    qv[r] = to_f32(qf2[it >> 1].p[0][(it & 1) * 4 + r]);
                }
                kv *= rk;
                qv *= rq;
                dq[it][n] += q1;
                dk[it][n] += A + be * F;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    qd[4 * it + r] += qv[r] * q1[r];
                    ka[4 * it + r] += kv[r] * A[r];
                    kf[4 * it + r] += kv[r] * F[r];
                    km[4 * it + r] += kv[r] * m3[r];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 16 * (i >> 2) + 4 * lg + (i & 3);
            const float x0 = group_allreduce<16>(qd[i]), x1 = group_allreduce<16>(ka[i]);
            const float x2 = group_allreduce<16>(kf[i]), x3 = group_allreduce<16>(km[i]);
            if (l16 == 0) {
                s.red[w][0][row] = x0;
                s.red[w][1][row] = x1;
                s.red[w][2][row] = x2;
                s.red[w][3][row] = x3;
            }
        }
        __syncthreads();
        if (w == 0) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = (s.red[0][i][lane] + s.red[1][i][lane]) + (s.red[2][i][lane] + s.red[3][i][lane]);
            const float be = s.tab[2 * 64 + lane];
            double dG = (double)x[0] + x[1] - (double)be * x[2];
            const double end = wave_sum((double)be * x[3]);
            if (lane == 63)
                dG += end + (double)__builtin_amdgcn_exp2f(s.tab[63]) * ((double)s.ip[0] + s.ip[1] + ((double)s.ip[2] + s.ip[3]));
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double dn = __shfl_down(dG, d);
                if (lane + d < 64) dG += dn;
            }
            if (lane < c.len) {
                const int64_t o = (c.tok + lane) * a.Hv + hv;
                a.dg[o] = (float)dG;
                a.dbeta[o] = x[2];
            }
            s.tq[lane] += x[0];
            s.tk[lane] += x[1] + be * x[2];
        }
    }
    __syncthreads();
    // with q = n scale and n = x rq / scale: dx = rq (dq - q (q . dq) / scale^2)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int kc = 16 * (NT * w + n) + l16;
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * it + 4 * lg + r;
                if (t >= c.len) continue;
                const float rq = s.tab[4 * 64 + t], rk = s.tab[3 * 64 + t];
                float x = dq[it][n][r] * rq, z = dk[it][n][r] * rk;
                if (a.norm) {
                    const float nq = rq / a.scale;   // 1 / |q|
                    x -= nq * nq * to_f32(s.qt[kc * LT + kpos(t)]) * s.tq[t];
                    z -= rk * rk * to_f32(s.kt[kc * LT + kpos(t)]) * s.tk[t];
                }
                const int64_t o = ((c.tok + t) * a.Hk + hk) * K + kc;
                a.dq[o] = (T)x;
                a.dk[o] = (T)z;
            }
    }
}

template <typename T, int K>
hipError_t launch_t(const Launch &a, hipStream_t stream)
{
    GradArgs<T> p;
    p.map = a.map;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.dy = static_cast<const T *>(a.dy);
    p.S = a.rec_s;
    p.E = a.rec_e;
    p.D = a.ws_ds;
    p.dR = a.ws_dr;
    p.table = a.table;
    p.dq = static_cast<T *>(a.dq);
    p.dk = static_cast<T *>(a.dk);
    p.dg = a.dg;
    p.dbeta = a.dbeta;
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.V = a.V;
    p.group = (int)(a.Hv / a.Hk);
    p.norm = a.norm;
    p.scale = a.scale;
    hipLaunchKernelGGL((gdr_grads_kernel<T, K>), dim3((unsigned)a.map.slots, (unsigned)a.Hk), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grads(const Launch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.K == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    return a.K == 64 ? launch_t<bf16, 64>(a, stream) : launch_t<bf16, 128>(a, stream);
}

}  // namespace gdr
}  // namespace wkv7
