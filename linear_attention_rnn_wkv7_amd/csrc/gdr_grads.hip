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
// One workgroup per chunk and key head; it adds up the group's value heads in
// registers.  Each of its K / 16 waves owns 16 key columns: it reads its rows
// of S and D once from memory as operands.  E, dR, dY pass through LDS 32
// values at a time, then Z and X, in operand order; so that two workgroups
// share a compute unit and cover each other's waits.

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

constexpr int kVB = 32;   // values of E, dR, dY in LDS at a time

template <typename T, int K>
struct GradLds {
    static constexpr int P = Num<T>::kPlanes, LV = kVB + kPad<T>, W = K / 16;
    char k[Swizzled<T, K>::kBytes], q[Swizzled<T, K>::kBytes];
    union {
        struct {
            T dy[64 * LV], dr[P * 64 * LV], e[P * 64 * LV];
        } in;
        T w[2][P * kTri];   // of Z, then of X: by rows, and transposed
    } u;
    float tab[kTableFloats], gam[64], eh[64];
    float red[4][W][64];       // q.dq, k.A, k.F, k.M3 of each wave's columns
    float ip[W];               // <S, D>
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

// Row and column of triangle tile t.
__device__ __forceinline__ int tile_row(int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; }

// Row sums over the wave's 16 columns of x * y, into red.
__device__ __forceinline__ void row_dots(float *red, int it, int lg, int l16, f32x4 x, f32x4 y)
{
    const f32x4 xy = x * y;
    f32x4 z;
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = group_allreduce<16>(xy[r]);
    if (l16 == 0) *reinterpret_cast<f32x4 *>(red + 16 * it + 4 * lg) = z;
}

template <typename T, int K, bool kShared>
__global__ void __launch_bounds__(4 * K, 2) gdr_grads_kernel(GradArgs<T> a)
{
    using L = GradLds<T, K>;
    using Quad = typename Num<T>::Quad;
    using Sw = Swizzled<T, K>;
    constexpr int P = L::P, LV = L::LV, W = L::W, NZ = (10 + W - 1) / W;   // tiles of Z, X per wave
    __shared__ __align__(16) char buf[sizeof(L)];
    L &s = *reinterpret_cast<L *>(buf);
    // the heads of a chunk together on one of the 8 dies, as in gdr_prep.hip: dg
    // and dbeta are a few bytes of each line to a head
    const int64_t at = blockIdx.x >> 3, slot = at / a.Hk * 8 + (blockIdx.x & 7), hk = at % a.Hk;
    if (slot >= a.map.slots) return;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, lg = lane >> 4, l16 = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

    if (w < 2) {
        dma_rows<T, K>(w ? s.q : s.k, (w ? a.q : a.k) + (c.tok * a.Hk + hk) * K, a.Hk * K, c.len, lane);
        wait_dma();
    }
    if (tid < 64) s.tq[tid] = s.tk[tid] = 0.f;

    f32x4 dq[4], dk[4];
    if constexpr (kShared) {
#pragma unroll
        for (int it = 0; it < 4; ++it) dq[it] = dk[it] = zero4();
    }
    for (int gi = 0; gi < (kShared ? a.group : 1); ++gi) {
        const int64_t hv = hk * a.group + gi, ch = slot * a.Hv + hv;
        __syncthreads();
        for (int i = tid; i < kTableFloats / 4; i += 64 * W)
            reinterpret_cast<f32x4 *>(s.tab)[i] = reinterpret_cast<const f32x4 *>(a.table + ch * kTableFloats)[i];
        f32x4 M1[4], M2[4], M3[4], Z[NZ], X[NZ];
        float ip = 0.f;
#pragma unroll
        for (int it = 0; it < 4; ++it) M1[it] = M2[it] = M3[it] = zero4();
#pragma unroll
        for (int i = 0; i < NZ; ++i) Z[i] = X[i] = zero4();
        const float *Sr = a.S + (ch * K + 16 * w + l16) * a.V + 4 * lg, *Dr = a.D + (ch * K + 16 * w + l16) * a.V + 4 * lg;
        for (int v0 = 0; v0 < (int)a.V; v0 += kVB) {
            // V is a multiple of 16: the second half of the block may be beyond it
            const bool half = v0 + 16 < (int)a.V;
            f32x4 x[2] = {zero4(), zero4()}, d[2] = {zero4(), zero4()};
            x[0] = *reinterpret_cast<const f32x4 *>(Sr + v0);
            d[0] = *reinterpret_cast<const f32x4 *>(Dr + v0);
            if (half) {
                x[1] = *reinterpret_cast<const f32x4 *>(Sr + v0 + 16);
                d[1] = *reinterpret_cast<const f32x4 *>(Dr + v0 + 16);
            }
            Quad yq[8 / W];
            f32x4 rq[8 / W], eq[8 / W];
#pragma unroll
            for (int n = 0; n < 8 / W; ++n) {
                const int t = (tid + n * 64 * W) >> 3, v = v0 + 4 * (tid & 7);
                yq[n] = Quad{};
                rq[n] = eq[n] = zero4();
                if (v < (int)a.V) {
                    if (t < c.len) yq[n] = *reinterpret_cast<const Quad *>(a.dy + ((c.tok + t) * a.Hv + hv) * a.V + v);
                    rq[n] = *reinterpret_cast<const f32x4 *>(a.dR + (ch * 64 + t) * a.V + v);
                    eq[n] = *reinterpret_cast<const f32x4 *>(a.E + (ch * 64 + t) * a.V + v);
                }
            }
            if (v0 > 0) __syncthreads();   // the block before is done with
#pragma unroll
            for (int n = 0; n < 8 / W; ++n) {
                const int at = ((tid + n * 64 * W) >> 3) * LV + kpos(4 * (tid & 7));
                Quad rz[P], ez[P];
                split_quad<T, P>(rq[n], rz);
                split_quad<T, P>(eq[n], ez);
                *reinterpret_cast<Quad *>(s.u.in.dy + at) = yq[n];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    *reinterpret_cast<Quad *>(s.u.in.dr + p * 64 * LV + at) = rz[p];
                    *reinterpret_cast<Quad *>(s.u.in.e + p * 64 * LV + at) = ez[p];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 xd = x[h] * d[h];
                ip += (xd[0] + xd[1]) + (xd[2] + xd[3]);
            }
            const Frag<T, P> Sf = make_frag<T, P>(x[0], x[1]), Df = make_frag<T, P>(d[0], d[1]);
            __syncthreads();
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                M1[it] = mma(M1[it], load_frag<T, 1>(s.u.in.dy, 16 * it + l16, LV, 0, lg, 0), Sf);
                M2[it] = mma(M2[it], load_frag<T, P>(s.u.in.dr, 16 * it + l16, LV, 0, lg, 64 * LV), Sf);
                M3[it] = mma(M3[it], load_frag<T, P>(s.u.in.e, 16 * it + l16, LV, 0, lg, 64 * LV), Df);
            }
            // tiles w, w + W, .. of Z, and from the other end of X
#pragma unroll
            for (int i = 0; i < NZ; ++i) {
                const int tz = w + i * W, tx = 9 - tz;
                if (tz >= 10) continue;
                const int zi = tile_row(tz), zj = tz - tile_id(zi, 0), xi = tile_row(tx), xj = tx - tile_id(xi, 0);
                Z[i] = mma(Z[i], load_frag<T, 1>(s.u.in.dy, 16 * zi + l16, LV, 0, lg, 0),
                           load_frag<T, P>(s.u.in.e, 16 * zj + l16, LV, 0, lg, 64 * LV));
                X[i] = mma(X[i], load_frag<T, P>(s.u.in.dr, 16 * xi + l16, LV, 0, lg, 64 * LV),
                           load_frag<T, P>(s.u.in.e, 16 * xj + l16, LV, 0, lg, 64 * LV));
            }
        }
        if (tid < 64) {
            s.gam[tid] = __builtin_amdgcn_exp2f(s.tab[tid] + s.tab[64 + tid]);
            s.eh[tid] = __builtin_amdgcn_exp2f((s.tab[63] - s.tab[tid]) + (s.tab[64 + 63] - s.tab[64 + tid]));
        }
        ip = wave_sum(ip);
        if (lane == 0) s.ip[w] = ip;
        // this wave's columns of q and k as operands; position 4 (it & 1) + r of
        // step it / 2 is row 16 it + 4 lg + r
        Frag<T, 1> kf[2], qf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            kf[ks] = Sw::cols(s.k, w, ks, lg, l16);
            qf[ks] = Sw::cols(s.q, w, ks, lg, l16);
        }
        auto value = [&](const Frag<T, 1> (&f)[2], int it, int kind) {
            f32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = to_f32(f[it >> 1].p[0][(it & 1) * 4 + r]);
            return x * row4(s.tab, kind, 16 * it + 4 * lg);
        };
        __syncthreads();   // E, dR, dY are done with; gam and eh are there
#pragma unroll
        for (int it = 0; it < 4; ++it) {   // now M1, M2, M3 become dq, A, F
            const f32x4 gam = row4(s.gam, 0, 16 * it + 4 * lg);
            M1[it] *= gam;
            M2[it] *= -gam;
            M3[it] *= row4(s.eh, 0, 16 * it + 4 * lg);
            row_dots(s.red[3][w], it, lg, l16, value(kf, it, 3), M3[it]);
        }
#pragma unroll
        for (int zx = 0; zx < 2; ++zx) {
            if (zx) __syncthreads();   // Z's operands are done with
#pragma unroll
            for (int n = 0; n < NZ; ++n) {   // with their decays, as operands
                const int t = zx ? 9 - (w + n * W) : w + n * W;
                if (w + n * W >= 10) continue;
                const int it = tile_row(t), jt = t - tile_id(it, 0), j = 16 * jt + l16, i0 = 16 * it + 4 * lg;
                const float Ghj = s.tab[j], Glj = s.tab[64 + j], cj = s.tab[2 * 64 + j] * s.tab[3 * 64 + j];   // beta rk
                const f32x4 gh = row4(s.tab, 0, i0), gl = row4(s.tab, 1, i0);
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float gd = __builtin_amdgcn_exp2f((gh[r] - Ghj) + (gl[r] - Glj));
                    x[r] = (zx ? i0 + r > j : i0 + r >= j) ? gd * (zx ? -X[n][r] : Z[n][r]) : 0.f;
                    // row i, k = j
                    put1<T, P>(s.u.w[0], tri_at<T, false>(t, (l16 >> 2) * 16 + 4 * lg + r) + (l16 & 3), x[r] * cj);
                }
                put<T, P>(s.u.w[1], tri_at<T, true>(t, lane), x * row4(s.tab, zx ? 3 : 4, i0));   // row j, k = i
            }
            __syncthreads();
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                f32x4 &m = zx ? M2[it] : M1[it];
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks) m = mma(m, load_tri<T, P, false>(s.u.w[0], it, ks, lane), kf[ks]);
#pragma unroll
                for (int ks = it / 2; ks < 2; ++ks)
                    M3[it] = mma(M3[it], load_tri<T, P, true>(s.u.w[1], it, ks, lane), zx ? kf[ks] : qf[ks]);
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const f32x4 kv = value(kf, it, 3);
            row_dots(s.red[0][w], it, lg, l16, value(qf, it, 4), M1[it]);
            row_dots(s.red[1][w], it, lg, l16, kv, M2[it]);
            row_dots(s.red[2][w], it, lg, l16, kv, M3[it]);
            M2[it] += row4(s.tab, 2, 16 * it + 4 * lg) * M3[it];
            if constexpr (kShared) {
                dq[it] += M1[it];
                dk[it] += M2[it];
            } else {
                dq[it] = M1[it];
                dk[it] = M2[it];
            }
        }
        __syncthreads();
        if (w == 0) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = 0.f;
#pragma unroll
                for (int n = 0; n < W; ++n) x[i] += s.red[i][n][lane];
            }
            const float be = s.tab[2 * 64 + lane];
            double dG = (double)x[0] + x[1] - (double)be * x[2];
            double end = wave_sum((double)be * x[3]), sd = 0.;
#pragma unroll
            for (int n = 0; n < W; ++n) sd += s.ip[n];
            end += (double)__builtin_amdgcn_exp2f(s.tab[63]) * sd;
            if (lane == 63) dG += end;
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
    if (a.norm) __syncthreads();
    // with q = n scale and n = x rq / scale: dx = rq (dq - q (q . dq) / scale^2)
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int t0 = 16 * it + 4 * lg;
        const f32x4 rq = row4(s.tab, 4, t0), rk = row4(s.tab, 3, t0);
        f32x4 x = dq[it] * rq, z = dk[it] * rk;
        if (a.norm) {
            const f32x4 nq = rq / a.scale, tq = row4(s.tq, 0, t0), tk = row4(s.tk, 0, t0);   // nq = 1 / |q|
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int b = (16 * w + l16) * (int)sizeof(T);
                x[r] -= nq[r] * nq[r] * to_f32(*reinterpret_cast<const T *>(s.q + Sw::at(t0 + r, b))) * tq[r];
                z[r] -= rk[r] * rk[r] * to_f32(*reinterpret_cast<const T *>(s.k + Sw::at(t0 + r, b))) * tk[r];
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (t0 + r >= c.len) continue;
            const int64_t o = ((c.tok + t0 + r) * a.Hk + hk) * K + 16 * w + l16;
            a.dq[o] = (T)x[r];
            a.dk[o] = (T)z[r];
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
    const dim3 grid((unsigned)((a.map.slots + 7) / 8 * 8 * a.Hk));
    if (p.group > 1)
        hipLaunchKernelGGL((gdr_grads_kernel<T, K, true>), grid, dim3(4 * K), 0, stream, p);
    else
        hipLaunchKernelGGL((gdr_grads_kernel<T, K, false>), grid, dim3(4 * K), 0, stream, p);
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
