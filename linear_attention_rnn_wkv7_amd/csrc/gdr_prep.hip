// Per chunk and value head: what the scans need besides q, k and v.
//
//   table [8][64], per token i of the chunk (rk, rq the reciprocal lengths of
//   k_i, q_i under GDR_NORM_QK, else 1; G the inclusive sum of g):
//     0  gamma_i rk             1  gamma_i rq scale
//     2  (gamma_C / gamma_i) rk beta_i
//     3  beta_i    4, 5  G_i log2(e) as a sum of two floats    6  rk    7  rq scale
//   tfrag: T = (I + N diag(beta))^-1,  pfrag: P (or their transposes), in
//   fragment order, as the parts the scans take.  q . k and k . k run once per key head on the matrix
//   cores; rk, rq and the decays are applied to the products, so that q and k
//   enter as they are.
//
// T is formed by forward substitution inside its four diagonal 16 x 16
// blocks (one lane per block and column), X_jj, and from those row by row of
// blocks, X_ij = -X_ii (sum_{k = j}^{i-1} L_ik X_kj), on fp32 matrix
// instructions.  (Powers of L would need fewer dependent steps, but for keys
// that are alike they grow like binomials and cancel.)
//
// One wave per chunk and key head: nothing waits at a barrier, and result
// tiles pass between the steps in registers; those that are needed as left
// operands go through 12.8 KB of LDS per wave.
//
// Tokens behind the sequence's end count as k = q = 0, g = 0, beta = 0.

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {
namespace {

// The ten 16 x 16 tiles of a lower triangle in LDS, rows 20 floats apart
// (16-byte reads of 16 rows meet all banks).
constexpr int kRow = 20, kTile = 16 * kRow;
__device__ __forceinline__ constexpr int tile_id(int i, int j) { return i * (i + 1) / 2 + j; }

struct WaveLds {
    float t[10 * kTile];
    float rq[64], rk[64], Gh[64], Gl[64], cb[64];
};

template <typename T>
struct PrepArgs {
    Map map;
    const T *q, *k;
    const float *g, *beta;
    float *table;
    T *tfrag, *pfrag;
    int64_t Hk, Hv;
    int group, norm;
    float scale;
};

__device__ __forceinline__ f32x4 mma16(f32x4 c, f32x4 a, f32x4 b)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

// A triangle's tiles (D layout) in fragment order, as P parts; `t` is the
// wave's LDS.
template <typename T, int P, bool kTrans>
__device__ __forceinline__ void write_frags(T *out, const f32x4 (&X)[10], float *t, int lane)
{
    const int lg = lane >> 4, l16 = lane & 15;
    if constexpr (!kTrans) {
#pragma unroll
        for (int i = 0; i < 10; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) t[i * kTile + (4 * lg + r) * kRow + l16] = X[i][r];
        wave_sync();
    }
#pragma unroll
    for (int f = 0; f < 6; ++f) {
        f32x4 half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (kTrans) {   // a result tile is its transpose's left operand
                const int jt = f < 4 ? f >> 1 : f - 2, it = 2 * (f < 4 ? f & 1 : 1) + h;
                half[h] = it < jt ? zero4() : X[tile_id(it < jt ? jt : it, jt)];
            } else {
                const int it = f < 2 ? f : (f + 2) >> 1, jt = 2 * (f < 2 ? 0 : f & 1) + h;
                half[h] = zero4();
                if (jt <= it)
                    half[h] = *reinterpret_cast<const f32x4 *>(t + tile_id(it, jt) * kTile + l16 * kRow + 4 * lg);
            }
        }
        const Frag<T, P> fr = make_frag<T, P>(half[0], half[1]);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<typename Num<T>::Oct *>(out + p * kFragElems + (f * 64 + lane) * 8) = fr.p[p];
    }
    if constexpr (!kTrans) wave_sync();
}

template <typename T, int K, bool kTrans>
__global__ void __launch_bounds__(256, 2) gdr_prep_kernel(PrepArgs<T> a)
{
    __shared__ __align__(16) WaveLds lds[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, lg = lane >> 4, l16 = lane & 15;
    WaveLds &s = lds[w];
    const int64_t slot = (int64_t)blockIdx.x * 4 + w, hk = blockIdx.y;
    if (slot >= a.map.slots) return;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;

    // the lower tiles of K K^T and Q K^T, straight from memory
    f32x4 kk[10], qk[10];
    float nq[4], nk[4];
#pragma unroll
    for (int i = 0; i < 10; ++i) kk[i] = qk[i] = zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) nq[i] = nk[i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        Frag<T, 1> fk[4], fq[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            fk[it].p[0] = fq[it].p[0] = typename Num<T>::Oct{};
            const int t = 16 * it + l16;
            if (t < c.len) {
                const int64_t o = ((c.tok + t) * a.Hk + hk) * K + 32 * ks + 8 * lg;
                fk[it].p[0] = *reinterpret_cast<const typename Num<T>::Oct *>(a.k + o);
                fq[it].p[0] = *reinterpret_cast<const typename Num<T>::Oct *>(a.q + o);
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                kk[tile_id(it, jt)] = mma(kk[tile_id(it, jt)], fk[it], fk[jt]);
                qk[tile_id(it, jt)] = mma(qk[tile_id(it, jt)], fq[it], fk[jt]);
            }
            if (a.norm) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    nq[it] += to_f32(fq[it].p[0][j]) * to_f32(fq[it].p[0][j]);
                    nk[it] += to_f32(fk[it].p[0][j]) * to_f32(fk[it].p[0][j]);
                }
            }
        }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        float x = a.scale, z = 1.f;
        if (a.norm) {
            nq[it] += __shfl_xor(nq[it], 16);
            nk[it] += __shfl_xor(nk[it], 16);
            nq[it] += __shfl_xor(nq[it], 32);
            nk[it] += __shfl_xor(nk[it], 32);
            x = a.scale / sqrtf(nq[it] + 1e-6f);
            z = 1.f / sqrtf(nk[it] + 1e-6f);
        }
        if (lg == 0) {
            s.rq[16 * it + l16] = x;
            s.rk[16 * it + l16] = z;
        }
    }
    wave_sync();
    const float rql = s.rq[lane], rkl = s.rk[lane];

    for (int gi = 0; gi < a.group; ++gi) {
        const int64_t hv = hk * a.group + gi, ch = slot * a.Hv + hv;
        {   // lane = token
            const bool in = lane < c.len;
            const int64_t o = (c.tok + (in ? lane : 0)) * a.Hv + hv;
            float g = in ? a.g[o] : 0.f;
            const float be = in ? a.beta[o] : 0.f;
            g = g < -200.f ? -200.f : g;   // exp is zero there; keeps differences finite
            double G = (double)g * 1.4426950408889634074;
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
            float *tb = a.table + ch * kTableFloats + lane;
            tb[0] = in ? ga * rkl : 0.f;
            tb[64] = in ? ga * rql : 0.f;
            tb[128] = in ? eh * rkl * be : 0.f;
            tb[192] = be;
            tb[256] = hi;
            tb[320] = lo;
            tb[384] = rkl;
            tb[448] = rql;
        }
        wave_sync();
        // L = N diag(beta) into LDS, P in registers
        f32x4 X[10], pp[10];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            const int j = 16 * jt + l16;
            const float Ghj = s.Gh[j], Glj = s.Gl[j], cj = s.cb[j];
#pragma unroll
            for (int it = jt; it < 4; ++it) {
                const int i0 = 16 * it + 4 * lg, id = tile_id(it, jt);
                const f32x4 gh = *reinterpret_cast<const f32x4 *>(s.Gh + i0), gl = *reinterpret_cast<const f32x4 *>(s.Gl + i0);
                const f32x4 rk = *reinterpret_cast<const f32x4 *>(s.rk + i0), rq = *reinterpret_cast<const f32x4 *>(s.rq + i0);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float gb = __builtin_amdgcn_exp2f((gh[r] - Ghj) + (gl[r] - Glj)) * cj;
                    const bool low = it > jt || 4 * lg + r > l16, diag = it == jt && 4 * lg + r == l16;
                    s.t[id * kTile + (4 * lg + r) * kRow + l16] = low ? kk[id][r] * rk[r] * gb : 0.f;
                    pp[id][r] = low || diag ? qk[id][r] * rq[r] * gb : 0.f;
                }
            }
        }
        wave_sync();
        {   // the diagonal blocks: lane (lg, l16) solves column l16 of block lg
            const float *L = s.t + tile_id(lg, lg) * kTile;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float acc = r == l16 ? 1.f : 0.f;
#pragma unroll
                for (int q4 = 0; q4 < r; q4 += 4) {
                    const f32x4 l = *reinterpret_cast<const f32x4 *>(L + r * kRow + q4);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q4 + q < r) acc = fmaf(-l[q], x[q4 + q], acc);
                }
                x[r] = acc;
            }
            wave_sync();
            float *D = s.t + tile_id(lg, lg) * kTile;
#pragma unroll
            for (int r = 0; r < 16; ++r) D[r * kRow + l16] = x[r];
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) X[tile_id(i, i)][r] = s.t[tile_id(i, i) * kTile + (4 * lg + r) * kRow + l16];
            if (i > 0) {
                const f32x4 xii = *reinterpret_cast<const f32x4 *>(s.t + tile_id(i, i) * kTile + l16 * kRow + 4 * lg);
                f32x4 li[3];
#pragma unroll
                for (int k = 0; k < i; ++k)
                    li[k] = *reinterpret_cast<const f32x4 *>(s.t + tile_id(i, k) * kTile + l16 * kRow + 4 * lg);
#pragma unroll
                for (int j = 0; j < i; ++j) {
                    f32x4 acc = zero4();
#pragma unroll
                    for (int k = j; k < i; ++k) acc = mma16(acc, li[k], X[tile_id(k, j)]);
                    X[tile_id(i, j)] = -mma16(zero4(), xii, acc);
                }
            }
        }
        wave_sync();
        constexpr int P = Num<T>::kPlanes, PP = kTrans ? P : kYParts<T>;
        write_frags<T, P, kTrans>(a.tfrag + ch * P * kFragElems, X, s.t, lane);
        write_frags<T, PP, kTrans>(a.pfrag + ch * PP * kFragElems, pp, s.t, lane);
    }
}

template <typename T, int K>
hipError_t launch_t(const Launch &a, bool transposed, hipStream_t stream)
{
    PrepArgs<T> p;
    p.map = a.map;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.g = a.g;
    p.beta = a.beta;
    p.table = a.table;
    p.tfrag = static_cast<T *>(a.tfrag);
    p.pfrag = static_cast<T *>(a.pfrag);
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.group = (int)(a.Hv / a.Hk);
    p.norm = a.norm;
    p.scale = a.scale;
    const dim3 grid((unsigned)((a.map.slots + 3) / 4), (unsigned)a.Hk);
    if (transposed)
        hipLaunchKernelGGL((gdr_prep_kernel<T, K, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((gdr_prep_kernel<T, K, false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_prep(const Launch &a, bool transposed, hipStream_t stream)
{
    if (a.dtype == WKV7_F32)
        return a.K == 64 ? launch_t<float, 64>(a, transposed, stream) : launch_t<float, 128>(a, transposed, stream);
    return a.K == 64 ? launch_t<bf16, 64>(a, transposed, stream) : launch_t<bf16, 128>(a, transposed, stream);
}

}  // namespace gdr
}  // namespace wkv7
