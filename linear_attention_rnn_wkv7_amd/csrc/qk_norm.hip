// The norm of queries and keys per head and their rotation, forward and
// backward.
//
// Bound by memory: D / 8 lanes to a head, 8 entries to a lane, each direction
// one pass.  A workgroup has a range of tokens; the angles of some of them are
// formed once, in fp64, and their cosines and sines kept in LDS for all heads.
// With n = x r w, r = 1 / sqrt(mean(x^2) + eps), and dn the gradient turned
// back by the same angle:
//     dx = r (dn w - x r m),  m = r mean(dn w x);   dw = sum dn x r
// Gradients of the weights are kept in registers over a workgroup's tokens and
// added up by a second kernel in a fixed order.
//
// 8 x 4096 tokens, 32 / 8 heads of 64, bf16: forward 73 us (4.6 TB/s), backward 103
// (4.9), the sum of the weights' 5.  One head at a time to a group of lanes instead
// of two has fewer loads in flight: 78 and 117.

#include <type_traits>

#include "attn_device.h"

namespace wkv7 {
namespace attn {
namespace {

constexpr int kAngles = 16;     // tokens whose angles are in LDS at a time

template <typename T>
struct NormArgs {
    const T *x[2];              // q, k
    const T *dz[2];
    T *out[2];                  // forward: z, backward: dx
    const float *w[2], *theta;
    const int32_t *positions;
    float *part;                // [parts][2][D]
    int64_t H[2], stride[2];
    int64_t T_, tokens, per;    // tokens of a workgroup
    int R, interleaved;
    float eps;
};

template <int L>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1) x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ float sum8(f32x8 x)
{
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}
template <typename T>
__device__ __forceinline__ f32x8 load8(const T *p)
{
    const Oct<T> x = *reinterpret_cast<const Oct<T> *>(p);
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __builtin_convertvector(x, f32x8);
}

// Turns a head's lane by its angles; dir -1 turns back.
template <int D>
__device__ __forceinline__ f32x8 turn(f32x8 x, const float *cs, const float *sn, int lane, int R, int interleaved,
                                      float dir)
{
    constexpr int L = D / 8;
    const int at = lane % L, col = 8 * at;
    if (interleaved) {
        if (col >= R) return x;
        f32x8 z;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = cs[col / 2 + j], s = dir * sn[col / 2 + j];
            z[2 * j] = x[2 * j] * c - x[2 * j + 1] * s;
            z[2 * j + 1] = x[2 * j + 1] * c + x[2 * j] * s;
        }
        return z;
    }
    const int apart = R / 16, first = at < apart;   // lanes between the two of a pair
    const int other = lane - at + (at < 2 * apart ? (first ? at + apart : at - apart) : at);
    f32x8 y;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __shfl(x[j], other);
    if (col >= R) return x;
    const int i = first ? col : col - R / 2;
    f32x8 z;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = x[j] * cs[i + j] + (first ? -dir : dir) * y[j] * sn[i + j];
    return z;
}

template <typename T, int D, bool kBackward>
__global__ void __launch_bounds__(256) qk_norm_kernel(NormArgs<T> a)
{
    constexpr int L = D / 8, N = 256 / L;   // heads at a time
    __shared__ float cs[kAngles][D / 2], sn[kAngles][D / 2];
    __shared__ float red[kBackward ? N : 1][D + 4];
    const int lane = threadIdx.x & 63, grp = threadIdx.x / L, col = 8 * (threadIdx.x % L);
    const int64_t begin = (int64_t)blockIdx.x * a.per;
    const int64_t end = begin + a.per < a.tokens ? begin + a.per : a.tokens;
    f32x8 dw[2];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
    for (int64_t t0 = begin; t0 < end; t0 += kAngles) {
        const int n = (int)(end - t0 < kAngles ? end - t0 : kAngles);
        if (a.theta) {
            __syncthreads();
            for (int i = threadIdx.x; i < n * (a.R / 2); i += 256) {
                const int t = i / (a.R / 2), p = i - t * (a.R / 2);
                const double pos = a.positions ? a.positions[t0 + t] : (double)((t0 + t) % a.T_);
                const double turns = pos * (double)a.theta[p] * 0.15915494309189533577;
                const float f = (float)(turns - rint(turns));   // of a whole turn, -1/2 to 1/2
                float s, c;
                sincospif(2.f * f, &s, &c);
                cs[t][p] = c;
                sn[t][p] = s;
            }
            __syncthreads();
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int H = (int)a.H[m];
            f32x8 w;
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (a.w[m]) w = load8(a.w[m] + col);
            // Heads i0 + grp, and N further, of these tokens.  Whole wavefronts take part:
            // heads behind the last repeat it.
            auto round = [&](int i0, auto count) __attribute__((always_inline)) {
                constexpr int U = decltype(count)::value;
                bool live[U];
                int t[U];
                int64_t to[U];
                f32x8 x[U], dz[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    live[u] = i0 + u * N + grp < n * H;
                    const int i = live[u] ? i0 + u * N + grp : n * H - 1;
                    t[u] = (uint32_t)i / (uint32_t)H;
                    const int h = i - t[u] * H;
                    const int64_t tok = t0 + t[u];
                    to[u] = (tok * H + h) * D + col;
                    x[u] = load8(a.x[m] + tok * a.stride[m] + (int64_t)h * D + col);
                    if constexpr (kBackward) dz[u] = load8(a.dz[m] + to[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float r = 1.f;
                    if (a.w[m]) r = 1.f / sqrtf(lanes_sum<L>(sum8(x[u] * x[u])) * (1.f / D) + a.eps);
                    f32x8 z;
                    if constexpr (!kBackward) {
                        z = x[u] * r * w;
                        if (a.theta) z = turn<D>(z, cs[t[u]], sn[t[u]], lane, a.R, a.interleaved, 1.f);
                    } else {
                        f32x8 dn = dz[u];
                        if (a.theta) dn = turn<D>(dn, cs[t[u]], sn[t[u]], lane, a.R, a.interleaved, -1.f);
                        z = dn;
                        if (a.w[m]) {
                            const f32x8 xn = x[u] * r;
                            if (live[u]) dw[m] += dn * xn;
                            dn *= w;
                            z = r * (dn - xn * (lanes_sum<L>(sum8(dn * xn)) * (1.f / D)));
                        }
                    }
                    if (live[u]) *reinterpret_cast<Oct<T> *>(a.out[m] + to[u]) = __builtin_convertvector(z, Oct<T>);
                }
            };
            int i0 = 0;
            for (; i0 + N < n * H; i0 += 2 * N) round(i0, std::integral_constant<int, 2>{});
            if (i0 < n * H) round(i0, std::integral_constant<int, 1>{});
        }
    }
    if constexpr (kBackward) {
        if (!a.part) return;
        for (int m = 0; m < 2; ++m) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) red[grp][col + j] = dw[m][j];
            __syncthreads();
            if (threadIdx.x < D) {
                float s = 0.f;
                for (int g = 0; g < N; ++g) s += red[g][threadIdx.x];
                a.part[((int64_t)blockIdx.x * 2 + m) * D + threadIdx.x] = s;
            }
        }
    }
}

// dw[m][col] = sum over the parts: a workgroup to 4 columns, 64 lanes to each,
// every 64th part to the same lane; then those, in order.
template <int D>
__global__ void __launch_bounds__(256) qk_norm_sum_kernel(const float *part, int64_t parts, float *dwq, float *dwk)
{
    __shared__ float red[64][5];
    const int col = threadIdx.x & 3, r = threadIdx.x >> 2;
    const int64_t at = (int64_t)blockIdx.x * 4 + col;
    float s = 0.f;
#pragma unroll 4
    for (int64_t i = r; i < parts; i += 64) s += part[i * 2 * D + at];
    red[r][col] = s;
    __syncthreads();
    if (r) return;
    s = 0.f;
#pragma unroll 8
    for (int i = 0; i < 64; ++i) s += red[i][col];
    (at < D ? dwq : dwk)[at % D] = s;
}

template <typename T, int D>
hipError_t launch_t(const QkNormLaunch &a, bool backward, hipStream_t stream)
{
    NormArgs<T> p;
    p.x[0] = static_cast<const T *>(a.q);
    p.x[1] = static_cast<const T *>(a.k);
    p.dz[0] = static_cast<const T *>(a.dqz);
    p.dz[1] = static_cast<const T *>(a.dkz);
    p.out[0] = static_cast<T *>(backward ? a.dq : a.qz);
    p.out[1] = static_cast<T *>(backward ? a.dk : a.kz);
    p.w[0] = a.wq;
    p.w[1] = a.wk;
    p.theta = a.theta;
    p.positions = a.positions;
    p.part = a.wq ? a.part : nullptr;
    p.H[0] = a.Hq;
    p.H[1] = a.Hk;
    p.stride[0] = a.q_stride;
    p.stride[1] = a.k_stride;
    p.T_ = a.T;
    p.tokens = a.B * a.T;
    // the forward leaves nothing to add up: as many workgroups as a compute unit holds
    const int64_t parts = backward ? qk_norm_parts(p.tokens) : p.tokens < 2048 ? p.tokens : 2048;
    p.per = (p.tokens + parts - 1) / parts;
    p.R = (int)a.R;
    p.interleaved = a.interleaved;
    p.eps = a.eps;
    if (!backward) {
        hipLaunchKernelGGL((qk_norm_kernel<T, D, false>), dim3((unsigned)parts), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((qk_norm_kernel<T, D, true>), dim3((unsigned)parts), dim3(256), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.wq) return e;
    hipLaunchKernelGGL((qk_norm_sum_kernel<D>), dim3(2 * D / 4), dim3(256), 0, stream, a.part, parts, a.dwq, a.dwk);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_forward(const QkNormLaunch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.D == 64 ? launch_t<float, 64>(a, false, stream) : launch_t<float, 128>(a, false, stream);
    return a.D == 64 ? launch_t<bf16, 64>(a, false, stream) : launch_t<bf16, 128>(a, false, stream);
}
hipError_t launch_qk_norm_backward(const QkNormLaunch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.D == 64 ? launch_t<float, 64>(a, true, stream) : launch_t<float, 128>(a, true, stream);
    return a.D == 64 ? launch_t<bf16, 64>(a, true, stream) : launch_t<bf16, 128>(a, true, stream);
}

}  // namespace attn
}  // namespace wkv7
