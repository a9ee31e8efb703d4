// Per chunk and value head: what the scans need besides q, k and v.
//
//   table [8][64], per token i of the chunk (rk, rq the reciprocal lengths of
//   k_i, q_i under GDR_NORM_QK, else 1; G the inclusive sum of g):
//     0  gamma_i rk             1  gamma_i rq scale
//     2  (gamma_C / gamma_i) rk beta_i
//     3  beta_i    4, 5  G_i as a sum of two floats    6  rk    7  rq scale
//   tfrag: T = (I + N diag(beta))^-1,  pfrag: P (or their transposes), in
//   fragment order.  q . k and k . k run once per key head on the matrix
//   cores; rk, rq and the decays are applied to the products, so that q and k
//   enter as they are.
//
// T is formed by forward substitution inside its four diagonal 16 x 16
// blocks, X_jj, and from those, block column by block column (one wave each),
// X_ij = -X_ii (sum_{k = j}^{i-1} L_ik X_kj) on fp32 matrix instructions.
// (Powers of L would need fewer dependent steps, but for keys that are alike
// they grow like binomials and cancel.)
//
// Tokens behind the sequence's end count as k = q = 0, g = 0, beta = 0.

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {
namespace {

constexpr int kLd = 68;   // fp32 64 x 64 arrays in LDS

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

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

__device__ __forceinline__ f32x4 mma16(f32x4 c, float4 a, f32x4 b)
{
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b[0], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b[1], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b[2], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b[3], c, 0, 0, 0);
    return c;
}

// Writes a 64 x 64 triangle (lower, or its transpose) in fragment order.
template <typename T, bool kTrans>
__device__ __forceinline__ void write_frags(T *out, const float *m, int tid)
{
    constexpr int P = Num<T>::kPlanes;
    for (int i = tid; i < 6 * 64; i += 256) {
        const int f = i >> 6, lane = i & 63, lg = lane >> 4, l16 = lane & 15;
        f32x4 lo, hi;
        if (!kTrans) {
            const int it = f < 2 ? f : (f + 2) >> 1, ks = f < 2 ? 0 : f & 1;
            const float *row = m + (16 * it + l16) * kLd + 32 * ks + 4 * lg;
            lo = *reinterpret_cast<const f32x4 *>(row);
            hi = *reinterpret_cast<const f32x4 *>(row + 16);
        } else {
            const int jt = f < 4 ? f >> 1 : f - 2, ks = f < 4 ? f & 1 : 1;
            const float *col = m + (32 * ks + 4 * lg) * kLd + 16 * jt + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                lo[r] = col[r * kLd];
                hi[r] = col[(16 + r) * kLd];
            }
        }
        const Frag<T, P> fr = make_frag<T, P>(lo, hi);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<typename Num<T>::Oct *>(out + p * kFragElems + i * 8) = fr.p[p];
    }
}

template <typename T, int K, bool kTrans>
__global__ void __launch_bounds__(256) gdr_prep_kernel(PrepArgs<T> a)
{
    constexpr int P = Num<T>::kPlanes;
    constexpr int LD = K + kPad<T>;
    constexpr int kOperands = 2 * 64 * LD * (int)sizeof(T), kSquares = 3 * 64 * kLd * 4;
    __shared__ __align__(16) char buf[kOperands > kSquares ? kOperands : kSquares];
    __shared__ float rq[64], rk[64], Gh[64], Gl[64], bt[64];
    T *sQ = reinterpret_cast<T *>(buf), *sK = sQ + 64 * LD;
    float *sL = reinterpret_cast<float *>(buf), *sX = sL + 64 * kLd, *sP = sX + 64 * kLd;

    const int64_t slot = blockIdx.x, hk = blockIdx.y;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, lg = lane >> 4, l16 = lane & 15;

    // q and k rows, and their lengths
    using Quad = typename Num<T>::Quad;
    for (int i = tid; i < 64 * (K / 4); i += 256) {
        const int t = i / (K / 4), col = 4 * (i % (K / 4));
        Quad x = {}, z = {};
        if (t < c.len) {
            const int64_t o = ((c.tok + t) * a.Hk + hk) * K + col;
            x = *reinterpret_cast<const Quad *>(a.q + o);
            z = *reinterpret_cast<const Quad *>(a.k + o);
        }
        *reinterpret_cast<Quad *>(sQ + t * LD + kpos(col)) = x;
        *reinterpret_cast<Quad *>(sK + t * LD + kpos(col)) = z;
        if (a.norm) {
            const f32x4 xf = quad_f32(x), zf = quad_f32(z);
            float sx = (xf[0] * xf[0] + xf[1] * xf[1]) + (xf[2] * xf[2] + xf[3] * xf[3]);
            float sz = (zf[0] * zf[0] + zf[1] * zf[1]) + (zf[2] * zf[2] + zf[3] * zf[3]);
            sx = group_allreduce<16>(sx);
            sz = group_allreduce<16>(sz);
            if (K == 128) {
                sx += __shfl_xor(sx, 16);
                sz += __shfl_xor(sz, 16);
            }
            if (col == 0) {
                rq[t] = a.scale / sqrtf(sx + 1e-6f);
                rk[t] = 1.f / sqrtf(sz + 1e-6f);
            }
        }
    }
    if (!a.norm && tid < 64) {
        rq[tid] = a.scale;
        rk[tid] = 1.f;
    }
    __syncthreads();

    // wave w: row tile w of K K^T and Q K^T
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero4();
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        const Frag<T, 1> ka = load_frag<T, 1>(sK, 16 * w + l16, LD, ks, lg, 0);
        const Frag<T, 1> qa = load_frag<T, 1>(sQ, 16 * w + l16, LD, ks, lg, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j <= w) {
                const Frag<T, 1> b = load_frag<T, 1>(sK, 16 * j + l16, LD, ks, lg, 0);
                kk[j] = mma(kk[j], ka, b);
                qk[j] = mma(qk[j], qa, b);
            }
        }
    }
    __syncthreads();   // q and k are done with

    for (int gi = 0; gi < a.group; ++gi) {
        const int64_t hv = hk * a.group + gi, ch = slot * a.Hv + hv;
        if (w == 0) {
            const bool in = lane < c.len;
            const int64_t o = (c.tok + (in ? lane : 0)) * a.Hv + hv;
            float g = in ? a.g[o] : 0.f;
            const float be = in ? a.beta[o] : 0.f;
            g = g < -200.f ? -200.f : g;   // exp is zero there; keeps differences finite
            double G = g;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double up = __shfl_up(G, d);
                if (lane >= d) G += up;
            }
            const double end = __shfl(G, 63);
            const float hi = (float)G, lo = (float)(G - (double)hi);
            const float ga = expf(hi), eh = expf((float)(end - G));
            Gh[lane] = hi;
            Gl[lane] = lo;
            bt[lane] = be;
            float *tb = a.table + ch * kTableFloats + lane;
            const float rkl = rk[lane], rql = rq[lane];
            const bool real = in;
            tb[0] = real ? ga * rkl : 0.f;
            tb[64] = real ? ga * rql : 0.f;
            tb[128] = real ? eh * rkl * be : 0.f;
            tb[192] = be;
            tb[256] = hi;
            tb[320] = lo;
            tb[384] = rkl;
            tb[448] = rql;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int jj = 16 * j + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * lg + r;
                float n = 0.f, p = 0.f;
                if (jj <= i) {
                    const float gb = expf((Gh[i] - Gh[jj]) + (Gl[i] - Gl[jj])) * bt[jj] * rk[jj];
                    n = jj < i ? kk[j][r] * rk[i] * gb : 0.f;
                    p = qk[j][r] * rq[i] * gb;
                }
                sL[i * kLd + jj] = n;
                sP[i * kLd + jj] = p;
                sX[i * kLd + jj] = 0.f;
            }
        }
        __syncthreads();
        {   // diagonal block w: lane l16 solves column l16
            const float *L = sL + 16 * w * kLd + 16 * w;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float acc = r == l16 ? 1.f : 0.f;
#pragma unroll
                for (int s = 0; s < r; ++s) acc = fmaf(-L[r * kLd + s], x[s], acc);
                x[r] = acc;
            }
            if (lg == 0) {
#pragma unroll
                for (int r = 0; r < 16; ++r) sX[(16 * w + r) * kLd + 16 * w + l16] = x[r];
            }
        }
        __syncthreads();
        {   // block column w
            f32x4 X[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i == w) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) X[i][r] = sX[(16 * i + 4 * lg + r) * kLd + 16 * w + l16];
                } else {
                    X[i] = zero4();
                }
                if (i > w) {
                    f32x4 acc = zero4();
#pragma unroll
                    for (int k = 0; k < i; ++k)
                        if (k >= w) acc = mma16(acc, ld4(sL + (16 * i + l16) * kLd + 16 * k + 4 * lg), X[k]);
                    f32x4 neg = mma16(zero4(), ld4(sX + (16 * i + l16) * kLd + 16 * i + 4 * lg), acc);
                    X[i] = -neg;
#pragma unroll
                    for (int r = 0; r < 4; ++r) sX[(16 * i + 4 * lg + r) * kLd + 16 * w + l16] = X[i][r];
                }
            }
        }
        __syncthreads();
        write_frags<T, kTrans>(a.tfrag + ch * P * kFragElems, sX, tid);
        write_frags<T, kTrans>(a.pfrag + ch * P * kFragElems, sP, tid);
        __syncthreads();
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
    const dim3 grid((unsigned)a.map.slots, (unsigned)a.Hk);
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
