// The recurrent form of the gated delta rule over a pool of states: for each
// row b, T tokens one after the other (T = 1 in a decode step, a few when
// drafted tokens are checked).
//
//     P = a S;  u = beta (v - P k);  S = P + u k^T;  y = scale S q
//
// A step reads and writes the whole V x K state for a few vectors, so it is
// bound by memory: each workgroup streams RPT passes of whole state rows
// through registers once, 16 bytes a lane, whatever T is.  16 KB of state per
// workgroup (64 rows of 64, 32 of 128) keeps a small batch spread over the
// chip: at 4 rows of 32 heads of 128 x 128 that is 512 workgroups.
// Measured: 256 rows of 32 heads of 64 x 64, fp32, 277 MB: 44 us, 6.3 TB/s
// (above a copy's rate: half of it stays in the last-level cache); 4 rows of
// 16 / 32 heads of 128 x 128, bf16, 17 MB: 7 us, most of it latency.  More tokens
// cost their chain of row sums: 4 tokens of each of the 256 rows 60 us; 8 of each
// of 64 rows of 16 / 32 heads of 128 x 128, bf16, 115 us for 285 MB.
//
// Thread t owns columns 4 (t mod TPR) .. of row m RPP + t / TPR, m < RPT; row
// dots are sums over the TPR lanes of a row in a fixed order.

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {
namespace {

template <typename T>
struct DecArgs {
    const T *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    T *y;
    int64_t T_, Hk, Hv, V, pool;
    int group, norm;
    float scale;
};

template <int TPR>
__device__ __forceinline__ float row_sum(float x)
{
    x = group_allreduce<16>(x);
    if (TPR == 32) x += __shfl_xor(x, 16);
    return x;
}

__device__ __forceinline__ float dot(f32x4 a, f32x4 b)
{
    return fmaf(a[3], b[3], fmaf(a[2], b[2], fmaf(a[1], b[1], a[0] * b[0])));
}

template <typename T, int K>
__global__ void __launch_bounds__(256) gdr_decode_kernel(DecArgs<T> p)
{
    constexpr int TPR = K / 4, RPP = 256 / TPR, RPT = 4;
    using Quad = typename Num<T>::Quad;
    const int t = threadIdx.x, col = 4 * (t % TPR);
    const int64_t b = blockIdx.z, hv = blockIdx.y, hk = hv / p.group;
    const int64_t row0 = (int64_t)blockIdx.x * RPP * RPT + t / TPR;
    const int64_t slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) return;
    float *st = p.state + ((slot * p.Hv + hv) * p.V + row0) * K + col;
    f32x4 S[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        S[m] = row0 + m * RPP < p.V ? *reinterpret_cast<const f32x4 *>(st + m * RPP * K) : zero4();
    if (p.slots) {   // an earlier row with this slot has it
        bool taken = false;
        for (int64_t i = t & 63; i < b; i += 64) taken |= p.slots[i] == slot;
        if (__any(taken)) return;
    }
    for (int64_t i = 0; i < p.T_; ++i) {
        const int64_t tok = b * p.T_ + i;
        f32x4 q = quad_f32(*reinterpret_cast<const Quad *>(p.q + (tok * p.Hk + hk) * K + col));
        f32x4 k = quad_f32(*reinterpret_cast<const Quad *>(p.k + (tok * p.Hk + hk) * K + col));
        const float a = expf(p.g[tok * p.Hv + hv]), be = p.beta[tok * p.Hv + hv];
        float sc = p.scale;
        if (p.norm) {
            sc /= sqrtf(row_sum<TPR>(dot(q, q)) + 1e-6f);
            k *= 1.f / sqrtf(row_sum<TPR>(dot(k, k)) + 1e-6f);
        }
        q *= sc;
#pragma unroll
        for (int m = 0; m < RPT; ++m) {
            const int64_t row = row0 + m * RPP;
            const int64_t o = (tok * p.Hv + hv) * p.V + row;
            const float v = row < p.V ? to_f32(p.v[o]) : 0.f;
            S[m] *= a;
            const float u = be * (v - row_sum<TPR>(dot(S[m], k)));
            S[m] += u * k;
            const float y = row_sum<TPR>(dot(S[m], q));
            if (col == 0 && row < p.V) p.y[o] = (T)y;
        }
    }
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        if (row0 + m * RPP < p.V) *reinterpret_cast<f32x4 *>(st + m * RPP * K) = S[m];
}

template <typename T, int K>
hipError_t launch_t(const DecodeLaunch &a, hipStream_t stream)
{
    DecArgs<T> p;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.v = static_cast<const T *>(a.v);
    p.g = a.g;
    p.beta = a.beta;
    p.state = a.state;
    p.slots = a.slots;
    p.y = static_cast<T *>(a.y);
    p.T_ = a.T;
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.V = a.V;
    p.pool = a.pool;
    p.group = (int)(a.Hv / a.Hk);
    p.norm = a.norm;
    p.scale = a.scale;
    const int64_t rows = 4 * 256 / (K / 4);
    hipLaunchKernelGGL((gdr_decode_kernel<T, K>),
                       dim3((unsigned)((a.V + rows - 1) / rows), (unsigned)a.Hv, (unsigned)a.B), dim3(256), 0,
                       stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeLaunch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.K == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    return a.K == 64 ? launch_t<bf16, 64>(a, stream) : launch_t<bf16, 128>(a, stream);
}

}  // namespace gdr
}  // namespace wkv7
