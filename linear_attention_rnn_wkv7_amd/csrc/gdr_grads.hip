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
//     dg_t = sum_{i >= t} gamma_i (q_i . M1_i - k_i . M2_i)
//          + sum_{i >= t > j} beta_j Gamma_ij (Z_ij q_i . k_j - X_ij k_i . k_j)
//          + sum_{j < t} beta_j e_j k_j . M3_j + gamma_C <S, D>
// Every term of dg_t has exp(g_t) as a factor.  (The gradients of the sums G,
// which are row dots of what dq and dk are made of, would give dg by a
// cumulative sum that needs no C x C array; but the terms without g_t cancel
// in it only but for their rounding, which at g = -16 is as large as dg.)
// Sums over i >= t and j < t run over a tile's registers and lanes, then its
// columns are added up; a wave has whole column tiles of Z and X, or, of eight
// waves, every other tile of one, which its sums over rows pass through.
//
// One workgroup per chunk and key head; it adds up the group's value heads in
// registers.  Each of its K / 16 waves owns 16 key columns: it reads its rows
// of S and D once from memory as operands.  E, dR, dY pass through LDS K / 2
// values at a time; then one copy each of the C x C arrays
//     U_ij = rq_i Gamma_ij Z_ij,   V_ij = -rk_i Gamma_ij X_ij
// (rq, rk: what q, k as passed are multiplied by), which serves by rows for dq
// and A, times rq_i and rk_i as the gradients of what was passed want them, and
// by columns for F.  By rows it meets k_j beta_j rk_j, by columns q and k as
// passed, exact in bf16.
//
// Measured, bf16: 8 x 4096 x 32, K = V = 64: 0.49 ms for 1.8 GB (3.6 TB/s); 4 x
// 4096 x 8 / 16 heads, K = V = 128: 0.42 ms for 1.0 GB; fp32, 8 x 4096 x 32, K = V =
// 64: 0.83 ms.  The time goes to turns of loading, LDS and products that at three
// and one workgroups to a compute unit overlap only in part: the matrix units are
// busy 0.25 and 0.21 of it, LDS waits for banks in 0.26 and 0.20.  dg without the
// cancelling sums took whole calls from 1091 to 1131 us at K = 128 and from 1123 to
// 1128 at K = 64.  When this form was chosen,
// loading the next block, or the next head's first, before the products did not
// help (443, 470 against 433 us at K = 128), values 64 at a time did (421), and S
// and D by [V][K] (413); two workgroups instead of three at K = 64 took 640 against
// 619 us.

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

// Rows of kVB values, their 16-byte pieces permuted so that 16 rows' reads of
// one piece meet all banks.
template <typename T>
__device__ __forceinline__ int in_row(int row, int k)   // of four values from k
{
    constexpr int kPer = 16 / (int)sizeof(T);   // values of a piece
    const int pos = kpos(k), piece = pos / kPer;
    return row * kVB + (piece ^ (sizeof(T) == 2 ? (row >> 2) & 3 : (row >> 1) & 7)) * kPer + pos % kPer;
}
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> load_in(const T *base, int it, int lg, int l16)
{
    Frag<T, P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const T *b = base + p * 64 * kVB;
        if constexpr (sizeof(T) == 2)
            f.p[p] = *reinterpret_cast<const typename Num<T>::Oct *>(b + in_row<T>(16 * it + l16, 4 * lg));
        else
            f.p[p] = __builtin_shufflevector(*reinterpret_cast<const f32x4 *>(b + in_row<T>(16 * it + l16, 4 * lg)),
                                             *reinterpret_cast<const f32x4 *>(b + in_row<T>(16 * it + l16, 16 + 4 * lg)),
                                             0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}

// A lower triangle's tiles, each stored by columns ([j][i], 16 x 16) per part.
constexpr int kTri16 = 10 * 256;
// Step ks of row tile `it` of the triangle itself (rows i, k = j).
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> tri_rows(const T *base, int it, int ks, int lg, int l16)
{
    Frag<T, P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        typename Num<T>::Quad h[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int jt = 2 * ks + n;
            h[n] = typename Num<T>::Quad{};
            if (jt > it) continue;
            const T *t = base + p * kTri16 + tile_id(it, jt) * 256;
            if constexpr (sizeof(T) == 2) {   // row j = 4 lg + l16 / 4, columns 4 (l16 % 4) .. to a lane
                const T *a = t + (4 * lg + (l16 >> 2)) * 16 + 4 * (l16 & 3);
                h[n] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (__attribute__((address_space(3))) bf16x4 *)(const __attribute__((address_space(3))) T *)a);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) h[n][r] = t[(4 * lg + r) * 16 + l16];
            }
        }
        f.p[p] = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}
// Step ks of row tile jt of its transpose (rows j, k = i).
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> tri_cols(const T *base, int jt, int ks, int lg, int l16)
{
    Frag<T, P> f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        typename Num<T>::Quad h[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int it = 2 * ks + n;
            h[n] = typename Num<T>::Quad{};
            if (it >= jt)
                h[n] = *reinterpret_cast<const typename Num<T>::Quad *>(base + p * kTri16 + tile_id(it, jt) * 256 + l16 * 16 + 4 * lg);
        }
        f.p[p] = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}

template <typename T, int K>
struct GradLds {
    static constexpr int P = Num<T>::kPlanes, W = K / 16, kBlocks = K / 64;   // blocks of values at a time
    char k[Swizzled<T, K>::kBytes], q[Swizzled<T, K>::kBytes];
    union {
        struct {
            T dy[64 * kVB], dr[P * 64 * kVB], e[P * 64 * kVB];
        } in[kBlocks];
        T w[2][P * kTri16];   // U, V
    } u;
    float tab[kTableFloats], gam[64], eh[64];
    float red[4][W][64];       // of each wave's columns: dg but for ip, k.F; with norm q.dq, k.A
    float ip[W];               // gamma_C <S, D>
    float tq[64], tk[64];      // over the group: q.dq, k.dk
};

// Row sums over the wave's 16 columns, into red.
__device__ __forceinline__ void row_sums(float *red, int it, int lg, int l16, f32x4 x)
{
    f32x4 z;
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = group_allreduce<16>(x[r]);
    if (l16 == 0) *reinterpret_cast<f32x4 *>(red + 16 * it + 4 * lg) = z;
}

// x[r] becomes the sum of x over a tile's rows from 4 lg + r on and `below`,
// which takes up the whole tile; column by column.
__device__ __forceinline__ f32x4 sums_from(f32x4 x, float &below, int lg)
{
    x[2] += x[3];
    x[1] += x[2];
    x[0] += x[1];
    const float a = __shfl_xor(x[0], 16), ab = x[0] + a, b = __shfl_xor(ab, 32);
    const float rest = ((lg & 1 ? 0.f : a) + (lg & 2 ? 0.f : b)) + below;
    below += ab + b;
    return x + rest;
}
// The same over the rows before 4 lg + r, and `above`.
__device__ __forceinline__ f32x4 sums_before(f32x4 x, float &above, int lg)
{
    const f32x4 z = {0.f, x[0], x[0] + x[1], (x[0] + x[1]) + x[2]};
    const float all = z[3] + x[3], a = __shfl_xor(all, 16), ab = all + a, b = __shfl_xor(ab, 32);
    const float rest = ((lg & 1 ? a : 0.f) + (lg & 2 ? b : 0.f)) + above;
    above += ab + b;
    return z + rest;
}

// Registers for three workgroups of four waves on a compute unit (LDS holds as
// many), or two where the sums over a group need them.
template <typename T, int K, bool kShared>
__global__ void __launch_bounds__(4 * K, K == 64 && sizeof(T) == 2 && !kShared ? 3 : 2) gdr_grads_kernel(GradArgs<T> a)
{
    using L = GradLds<T, K>;
    using Quad = typename Num<T>::Quad;
    using Sw = Swizzled<T, K>;
    constexpr int P = L::P, W = L::W, NB = L::kBlocks;
    __shared__ __align__(16) char buf[sizeof(L)];
    L &s = *reinterpret_cast<L *>(buf);
    // the heads of a chunk together on one of the 8 dies, as in gdr_prep.hip: dg
    // and dbeta are a few bytes of each line to a head
    const int64_t at = blockIdx.x >> 3, slot = at / a.Hk * 8 + (blockIdx.x & 7), hk = at % a.Hk;
    if (slot >= a.map.slots) return;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // column tile w % 4 of Z and 3 - w % 4 of X is this wave's, five tiles; of
    // eight waves, two have every other row tile
    constexpr int kHalf = W / 4;
    const int zcol = w & 3, xcol = 3 - zcol;
    auto mine = [&](int it, int jt) { return it >= jt && (kHalf == 1 || ((it ^ w ^ (w >> 2)) & 1) == 0); };

    if (w < 2) {
        dma_rows<T, K>(w ? s.q : s.k, (w ? a.q : a.k) + (c.tok * a.Hk + hk) * K, a.Hk * K, c.len, lane);
    }
    if (tid < 64) s.tq[tid] = s.tk[tid] = 0.f;

    f32x4 dq[4], dk[4];
    if constexpr (kShared) {
#pragma unroll
        for (int it = 0; it < 4; ++it) dq[it] = dk[it] = zero4();
    }
    for (int gi = 0; gi < (kShared ? a.group : 1); ++gi) {
        const int64_t hv = hk * a.group + gi, ch = slot * a.Hv + hv;
        f32x4 M1[4], M2[4], M3[4], Z[2][4 / kHalf];
        float ip = 0.f;
#pragma unroll
        for (int it = 0; it < 4; ++it) M1[it] = M2[it] = M3[it] = Z[0][it / kHalf] = Z[1][it / kHalf] = zero4();
        // addresses as a uniform base and 32-bit offsets
        const uint32_t V = (uint32_t)a.V;
        const float *Sb = a.S + ch * K * a.V, *Db = a.D + ch * K * a.V, *Rb = a.dR + ch * 64 * a.V, *Eb = a.E + ch * 64 * a.V;
        const T *yb = a.dy + (c.tok * a.Hv + hv) * a.V;
        const uint32_t ys = (uint32_t)(a.Hv * a.V);
        const f32x4 tv = reinterpret_cast<const f32x4 *>(a.table + ch * kTableFloats)[tid < kTableFloats / 4 ? tid : 0];
        if (gi > 0) __syncthreads();   // the table of the head before is done with
        for (uint32_t v0 = 0; v0 < V; v0 += NB * kVB) {
            // addresses formed anew, not kept
            const uint32_t ft = fresh((uint32_t)tid), lg = ft >> 4 & 3, l16 = ft & 15;
            // V is a multiple of 16: halves of the last block may be beyond it
            f32x4 x[NB][2], d[NB][2], rq[NB][8 / W], eq[NB][8 / W];
            Quad yq[NB][8 / W];
#pragma unroll
            for (int h = 0; h < 2 * NB; ++h) {
                const uint32_t so = (v0 + 16 * h + 4 * lg) * K + 16 * w + l16;
                f32x4 &xh = x[h >> 1][h & 1], &dh = d[h >> 1][h & 1];
                xh = dh = zero4();
                if (v0 + 16 * h < V) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        xh[j] = Sb[so + j * K];
                        dh[j] = Db[so + j * K];
                    }
                }
            }
            // NB = 2: 16 lanes to a row of both blocks
#pragma unroll
            for (int n = 0; n < NB * 8 / W; ++n) {
                const uint32_t t = (ft + n * 64 * W) / (8 * NB), v = v0 + 4 * (ft % (8 * NB));
                Quad &yn = yq[n / (8 / W)][n % (8 / W)];
                f32x4 &rn = rq[n / (8 / W)][n % (8 / W)], &en = eq[n / (8 / W)][n % (8 / W)];
                yn = Quad{};
                rn = en = zero4();
                if (v < V) {
                    if ((int)t < c.len) yn = *reinterpret_cast<const Quad *>(yb + t * ys + v);
                    rn = *reinterpret_cast<const f32x4 *>(Rb + t * V + v);
                    en = *reinterpret_cast<const f32x4 *>(Eb + t * V + v);
                }
            }
            if (v0 > 0)
                __syncthreads();   // the blocks before are done with
            else if (tid < kTableFloats / 4)
                reinterpret_cast<f32x4 *>(s.tab)[tid] = tv;
#pragma unroll
            for (int n = 0; n < NB * 8 / W; ++n) {
                const int to = in_row<T>((ft + n * 64 * W) / (8 * NB), 4 * (ft & 7));
                auto &in = s.u.in[NB == 1 ? 0 : ft >> 3 & 1];
                Quad rz[P], ez[P];
                split_quad<T, P>(rq[n / (8 / W)][n % (8 / W)], rz);
                split_quad<T, P>(eq[n / (8 / W)][n % (8 / W)], ez);
                *reinterpret_cast<Quad *>(in.dy + to) = yq[n / (8 / W)][n % (8 / W)];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    *reinterpret_cast<Quad *>(in.dr + p * 64 * kVB + to) = rz[p];
                    *reinterpret_cast<Quad *>(in.e + p * 64 * kVB + to) = ez[p];
                }
            }
            if (v0 == 0 && gi == 0) wait_dma();   // of k, q, older than the block's loads
            __syncthreads();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const auto &in = s.u.in[b];
                f32x4 xd = x[b][0] * d[b][0];
                xd += x[b][1] * d[b][1];
                ip += (xd[0] + xd[1]) + (xd[2] + xd[3]);
                // one array of rows after the other: registers for few operands at a time
                const Frag<T, P> Sf = make_frag<T, P>(x[b][0], x[b][1]);
                {
                    const Frag<T, P> E = load_in<T, P>(in.e, zcol, lg, l16);
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const Frag<T, 1> y = load_in<T, 1>(in.dy, it, lg, l16);
                        M1[it] = mma(M1[it], y, Sf);
                        if (mine(it, zcol)) Z[0][it / kHalf] = mma(Z[0][it / kHalf], y, E);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                {
                    const Frag<T, P> E = load_in<T, P>(in.e, xcol, lg, l16);
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const Frag<T, P> r = load_in<T, P>(in.dr, it, lg, l16);
                        M2[it] = mma(M2[it], r, Sf);
                        if (mine(it, xcol)) Z[1][it / kHalf] = mma(Z[1][it / kHalf], r, E);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                const Frag<T, P> Df = make_frag<T, P>(d[b][0], d[b][1]);
#pragma unroll
                for (int it = 0; it < 4; ++it) M3[it] = mma(M3[it], load_in<T, P>(in.e, it, lg, l16), Df);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        const int ln = (int)fresh(lane), lg = ln >> 4, l16 = ln & 15;
        if (tid < 64) {
            s.gam[tid] = __builtin_amdgcn_exp2f(s.tab[tid] + s.tab[64 + tid]);
            s.eh[tid] = __builtin_amdgcn_exp2f((s.tab[63] - s.tab[tid]) + (s.tab[64 + 63] - s.tab[64 + tid]));
        }
        // this wave's columns of q and k as operands; position 4 (it & 1) + r of
        // step it / 2 is row 16 it + 4 lg + r
        Frag<T, 1> kf[2], qf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            kf[ks] = Sw::cols(s.k, w, ks, lg, l16);
            qf[ks] = Sw::cols(s.q, w, ks, lg, l16);
        }
        auto value = [&](const Frag<T, 1> (&f)[2], int it) {
            f32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = to_f32(f[it >> 1].p[0][(it & 1) * 4 + r]);
            return x;
        };
        __syncthreads();   // E, dR, dY are done with; gam and eh are there
        f32x4 dg[4];   // row by row, of this wave's columns
#pragma unroll
        for (int it = 0; it < 4; ++it) dg[it] = zero4();
#pragma unroll
        for (int zx = 0; zx < 2; ++zx) {   // U and V
            const int jt = zx ? xcol : zcol, j = 16 * jt + l16;
            const float Ghj = s.tab[j], Glj = s.tab[64 + j], cj = s.tab[2 * 64 + j] * s.tab[3 * 64 + j];
            float below = 0.f;
#pragma unroll
            for (int it = 3; it >= 0; --it) {
                if (it < jt) continue;
                f32x4 x = zero4();
                if (mine(it, jt)) {
                    const int i0 = 16 * it + 4 * lg;
                    const f32x4 gh = row4(s.tab, 0, i0), gl = row4(s.tab, 1, i0), f = row4(s.tab, zx ? 3 : 4, i0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float gd = __builtin_amdgcn_exp2f((gh[r] - Ghj) + (gl[r] - Glj)) * f[r];
                        x[r] = (zx ? i0 + r > j : i0 + r >= j) ? gd * (zx ? -Z[1][it / kHalf][r] : Z[0][it / kHalf][r]) : 0.f;
                    }
                    Quad q[P];
                    split_quad<T, P>(x, q);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        *reinterpret_cast<Quad *>(s.u.w[zx] + p * kTri16 + tile_id(it, jt) * 256 + l16 * 16 + 4 * lg) = q[p];
                    f32x4 qk = zero4();   // q . k or k . k, as passed
#pragma unroll
                    for (int ks = 0; ks < K / 32; ++ks)
                        qk = mma(qk, Sw::rows(zx ? s.k : s.q, it, ks, lg, l16), Sw::rows(s.k, jt, ks, lg, l16));
                    x *= qk * cj;
                }
                const f32x4 sum = sums_from(x, below, lg);
#pragma unroll
                for (int r = 0; r < 4; ++r) dg[it][r] += it > jt || 4 * lg + r > l16 ? sum[r] : 0.f;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // M1, M2, M3 become rq dq, rk A, F
        f32x4 ck[4];
        float below = 0.f, above = 0.f;
#pragma unroll
        for (int it = 3; it >= 0; --it) {
            const int i0 = 16 * it + 4 * lg;
            const f32x4 gam = row4(s.gam, 0, i0);
            M1[it] *= gam * row4(s.tab, 4, i0);
            M2[it] *= -gam * row4(s.tab, 3, i0);
            dg[it] += sums_from(value(qf, it) * M1[it] + value(kf, it) * M2[it], below, lg);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i0 = 16 * it + 4 * lg;
            M3[it] *= row4(s.eh, 0, i0);
            ck[it] = value(kf, it) * (row4(s.tab, 2, i0) * row4(s.tab, 3, i0));
            row_sums(s.red[0][w], it, lg, l16, dg[it] + sums_before(ck[it] * M3[it], above, lg));
        }
        const Frag<T, P> cf[2] = {make_frag<T, P>(ck[0], ck[1]), make_frag<T, P>(ck[2], ck[3])};
        ip = wave_sum(ip * __builtin_amdgcn_exp2f(s.tab[63]));
        if (lane == 0) s.ip[w] = ip;
        __syncthreads();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks <= it / 2; ++ks) {
                M1[it] = mma(M1[it], tri_rows<T, P>(s.u.w[0], it, ks, lg, l16), cf[ks]);
                M2[it] = mma(M2[it], tri_rows<T, P>(s.u.w[1], it, ks, lg, l16), cf[ks]);
            }
#pragma unroll
            for (int ks = it / 2; ks < 2; ++ks) {
                M3[it] = mma(M3[it], tri_cols<T, P>(s.u.w[0], it, ks, lg, l16), qf[ks]);
                M3[it] = mma(M3[it], tri_cols<T, P>(s.u.w[1], it, ks, lg, l16), kf[ks]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i0 = 16 * it + 4 * lg;
            const f32x4 be = row4(s.tab, 2, i0), rk = row4(s.tab, 3, i0);
            const f32x4 kv = value(kf, it);
            row_sums(s.red[1][w], it, lg, l16, kv * rk * M3[it]);
            if (a.norm) {
                row_sums(s.red[2][w], it, lg, l16, value(qf, it) * M1[it]);   // q rq . dq
                row_sums(s.red[3][w], it, lg, l16, kv * M2[it]);
            }
            M2[it] += be * rk * M3[it];
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
                for (int n = 0; n < W; ++n) x[i] += i >= 2 && !a.norm ? 0.f : s.red[i][n][lane];
            }
            float all = 0.f;
#pragma unroll
            for (int n = 0; n < W; ++n) all += s.ip[n];
            if (lane < c.len) {
                const int64_t o = (c.tok + lane) * a.Hv + hv;
                a.dg[o] = x[0] + all;
                a.dbeta[o] = x[1];
            }
            s.tq[lane] += x[2];
            s.tk[lane] += x[3] + s.tab[2 * 64 + lane] * x[1];
        }
    }
    __syncthreads();
    const int ln = (int)fresh(lane), lg = ln >> 4, l16 = ln & 15;
    // with q = n scale and n = x rq / scale: dx = rq dq - x (rq / scale)^2 (q . dq),
    // each value in the place of the q or k that it needs, then out by whole rows
    const float is = 1.f / a.scale;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int t0 = 16 * it + 4 * lg;
        const f32x4 rq = row4(s.tab, 4, t0), rk = row4(s.tab, 3, t0);
        f32x4 x = dq[it], z = dk[it];
        f32x4 nq = rq * is, nk = rk;   // 1 / |q|, 1 / |k|
        nq *= nq * row4(s.tq, 0, t0);
        nk *= nk * row4(s.tk, 0, t0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int o = Sw::at(t0 + r, (16 * w + l16) * (int)sizeof(T));
            T *qs = reinterpret_cast<T *>(s.q + o), *ks = reinterpret_cast<T *>(s.k + o);
            if (a.norm) {
                x[r] -= nq[r] * to_f32(*qs);
                z[r] -= nk[r] * to_f32(*ks);
            }
            *qs = (T)x[r];
            *ks = (T)z[r];
        }
    }
    __syncthreads();
    T *dqb = a.dq + (c.tok * a.Hk + hk) * K, *dkb = a.dk + (c.tok * a.Hk + hk) * K;
    constexpr int kRow = K * (int)sizeof(T) / 16;   // 16-byte pieces of a row
#pragma unroll
    for (int n = 0; n < 64 * kRow / (64 * W); ++n) {
        const int i = tid + n * 64 * W, t = i / kRow, b = i % kRow * 16;
        if (t >= c.len) continue;
        const uint32_t o = (uint32_t)t * (uint32_t)(a.Hk * K) + b / sizeof(T);
        *reinterpret_cast<f32x4 *>(dqb + o) = *reinterpret_cast<const f32x4 *>(s.q + Sw::at(t, b));
        *reinterpret_cast<f32x4 *>(dkb + o) = *reinterpret_cast<const f32x4 *>(s.k + Sw::at(t, b));
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
    const dim3 grid((unsigned)grads_blocks(a.map.slots, a.Hk));
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
