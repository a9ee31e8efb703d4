// The norms around a recurrence: the epilogue of the gated delta rule (a
// gated root-mean-square norm of each head) and the residual norm between
// two blocks, forward and backward.
//
// Both are bound by memory: each direction reads its inputs and writes its
// outputs once, 8 values (16 or 32 bytes) per lane and access.  The backward
// of a norm needs two row sums, of x^2 and of dh w x; both are sums of
// what has been loaded, so one exchange between the row's lanes serves both:
//     r = 1 / sqrt(mean(x^2) + eps),  m = r mean(dh w x)
//     dx = r (dh w - x r m),          dw = sum over rows of dh x r
// Gradients of the weights are kept in registers over a workgroup's rows and
// added up by a second kernel in a fixed order.
//
// Measured, bf16: epilogue at 8 x 4096 x 32 heads of 64: forward 82 us for 403
// MB (4.9 TB/s), backward 128 us for 671 MB (5.2) and 15 us for the sums;
// residual norm at 32768 rows of 2048: forward 95 us for 537 MB (5.7 TB/s),
// backward with scale 170 us for 805 MB (4.7) and 2 x 7 us.  bf16 rows whose
// length is no multiple of 8 go by 2 bytes a lane: at 2047 and 2050 forward 204
// and 340 us (2.6 and 1.6 TB/s), backward with scale 928 and 992 us (0.9 and 0.8).

#include "gdr_device.h"

namespace wkv7 {
namespace gdr {
namespace {

__device__ __forceinline__ f32x8 load8(const float *p) { return *reinterpret_cast<const f32x8 *>(p); }
__device__ __forceinline__ f32x8 load8(const bf16 *p)
{
    return __builtin_convertvector(*reinterpret_cast<const bf16x8 *>(p), f32x8);
}
__device__ __forceinline__ void store8(float *p, f32x8 x) { *reinterpret_cast<f32x8 *>(p) = x; }
__device__ __forceinline__ void store8(bf16 *p, f32x8 x)
{
    *reinterpret_cast<bf16x8 *>(p) = __builtin_convertvector(x, bf16x8);
}
__device__ __forceinline__ float sum8(f32x8 x)
{
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}
__device__ __forceinline__ f32x8 zero8() { return f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}; }

// Sum over aligned groups of L lanes, in every lane.
template <int L>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// The most workgroups of a launch: its threads stay below 2^32.
constexpr int64_t max_blocks(int threads) { return (int64_t(1) << 32) / threads - 1; }

// ------------------------------------------------------------- the epilogue

template <typename T>
struct EpiArgs {
    const T *y, *gate, *dz;
    const float *w;
    T *z, *dy, *dgate;
    float *part;              // [Hw][parts][N]
    int64_t rows, H, Hw;      // heads of the forward's launch, tokens of the backward
    int64_t per, parts;       // rows of a weight head per backward workgroup
    float eps;
};

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <typename T, int N>
__global__ void __launch_bounds__(256) epilogue_fwd_kernel(EpiArgs<T> a)
{
    constexpr int L = N / 8, R = 256 / L;   // lanes per row, rows per workgroup
    const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / L;
    if (row >= a.rows) return;              // whole rows
    const int col = 8 * (threadIdx.x % L);
    const int64_t o = row * N + col;
    const f32x8 y = load8(a.y + o), g = load8(a.gate + o);
    const f32x8 w = load8(a.w + (a.Hw == 1 ? 0 : row % a.H * N) + col);
    const float r = 1.f / sqrtf(lanes_sum<L>(sum8(y * y)) * (1.f / N) + a.eps);
    f32x8 z;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[i] * r * w[i] * (g[i] * sigmoid(g[i]));
    store8(a.z + o, z);
}

// Workgroup (part, hw): rows part * per .. of the weight head's rows * H / Hw.
template <typename T, int N>
__global__ void __launch_bounds__(256) epilogue_bwd_kernel(EpiArgs<T> a)
{
    constexpr int L = N / 8, R = 256 / L;
    __shared__ float red[R][N + 4];
    const int col = 8 * (threadIdx.x % L), grp = threadIdx.x / L;
    const int64_t hw = blockIdx.y, all = a.rows * a.H / a.Hw;
    const int64_t end = (int64_t)(blockIdx.x + 1) * a.per < all ? (int64_t)(blockIdx.x + 1) * a.per : all;
    const f32x8 w = load8(a.w + hw * N + col);
    f32x8 dw = zero8();
    for (int64_t i = (int64_t)blockIdx.x * a.per + grp; i < end; i += R) {
        const int64_t o = (a.Hw == 1 ? i : i * a.H + hw) * N + col;
        const f32x8 y = load8(a.y + o), g = load8(a.gate + o), dz = load8(a.dz + o);
        f32x8 dn, sg;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sg[j] = sigmoid(g[j]);
            dn[j] = dz[j] * g[j] * sg[j];
        }
        const float r = 1.f / sqrtf(lanes_sum<L>(sum8(y * y)) * (1.f / N) + a.eps);
        const float m = lanes_sum<L>(sum8(dn * w * y)) * (1.f / N) * r;
        f32x8 dy, dg;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float yn = y[j] * r;
            dg[j] = dz[j] * yn * w[j] * sg[j] * (1.f + g[j] * (1.f - sg[j]));
            dy[j] = r * (dn[j] * w[j] - yn * m);
            dw[j] += dn[j] * yn;
        }
        store8(a.dgate + o, dg);
        store8(a.dy + o, dy);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) red[grp][col + j] = dw[j];
    __syncthreads();
    for (int j = threadIdx.x; j < N; j += 256) {
        float s = 0.f;
        for (int q = 0; q < R; ++q) s += red[q][j];
        a.part[(hw * a.parts + blockIdx.x) * N + j] = s;
    }
}

// out[g][j] = sum over p of part[g][p][j] for j < n: one workgroup per 64
// columns, 16 waves each adding every 16th part, then the 16 sums in order.
__global__ void __launch_bounds__(1024) parts_kernel(const float *part, float *out, int64_t parts, int64_t n,
                                                     int64_t part_stride, int64_t group_stride)
{
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t j = (int64_t)blockIdx.x * 64 + lane, g = blockIdx.y;
    float s = 0.f;
    if (j < n) {
#pragma unroll 4
        for (int64_t p = w; p < parts; p += 16) s += part[g * group_stride + p * part_stride + j];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && j < n) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 16; ++q) s += red[q][lane];
        out[g * n + j] = s;
    }
}

template <typename T, int N>
hipError_t epilogue_t(const EpilogueLaunch &a, bool backward, hipStream_t stream)
{
    EpiArgs<T> p;
    p.y = static_cast<const T *>(a.y);
    p.gate = static_cast<const T *>(a.gate);
    p.dz = static_cast<const T *>(a.dz);
    p.w = a.w;
    p.z = static_cast<T *>(a.z);
    p.dy = static_cast<T *>(a.dy);
    p.dgate = static_cast<T *>(a.dgate);
    p.part = a.part;
    p.rows = a.rows;
    p.H = a.H;
    p.Hw = a.Hw;
    p.eps = a.eps;
    constexpr int R = 256 / (N / 8);
    if (!backward) {
        // heads of a launch; with a weight for each of H (65535 at most), whole tokens
        const int64_t most = max_blocks(256) * R / a.Hw * a.Hw;
        for (int64_t left = a.rows * a.H; left > 0; left -= most) {
            p.rows = left < most ? left : most;
            hipLaunchKernelGGL((epilogue_fwd_kernel<T, N>), dim3((unsigned)((p.rows + R - 1) / R)), dim3(256), 0, stream,
                               p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            p.y += most * N;
            p.gate += most * N;
            p.z += most * N;
        }
        return hipSuccess;
    }
    const int64_t all = a.rows * a.H / a.Hw;
    p.parts = epilogue_parts(a.rows, a.H, N, a.Hw);
    p.per = (all + p.parts - 1) / p.parts;
    hipLaunchKernelGGL((epilogue_bwd_kernel<T, N>), dim3((unsigned)p.parts, (unsigned)a.Hw), dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(parts_kernel, dim3((N + 63) / 64, (unsigned)a.Hw), dim3(1024), 0, stream, a.part, a.dw,
                       p.parts, (int64_t)N, (int64_t)N, p.parts * N);
    return hipGetLastError();
}

template <typename T>
hipError_t epilogue_n(const EpilogueLaunch &a, bool backward, hipStream_t stream)
{
    switch (a.N) {
    case 16: return epilogue_t<T, 16>(a, backward, stream);
    case 32: return epilogue_t<T, 32>(a, backward, stream);
    case 64: return epilogue_t<T, 64>(a, backward, stream);
    case 128: return epilogue_t<T, 128>(a, backward, stream);
    default: return epilogue_t<T, 256>(a, backward, stream);
    }
}

// -------------------------------------------------------- the residual norm

template <typename T>
struct NormArgs {
    const T *x, *y, *dh, *dxo;
    const float *scale, *w;
    T *xo, *h, *dx, *dy;
    float *part;             // [parts][1 or 2][D]
    int64_t rows, per;       // rows per backward workgroup
    int D;
    float eps;
};

// The row's values of one thread: 8 at a time, kN times, NT threads apart;
// with kVec they are contiguous and D a multiple of 8, else NT apart.
template <int NT, bool kVec>
__device__ __forceinline__ int elem(int i, int j, int t)
{
    return kVec ? (i * NT + t) * 8 + j : (i * 8 + j) * NT + t;
}
template <typename T, int NT, bool kVec>
__device__ __forceinline__ f32x8 get8(const T *row, int i, int t, int D)
{
    f32x8 x = zero8();
    if (kVec) {
        if (elem<NT, true>(i, 0, t) < D) x = load8(row + elem<NT, true>(i, 0, t));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (elem<NT, false>(i, j, t) < D) x[j] = to_f32(row[elem<NT, false>(i, j, t)]);
    }
    return x;
}
template <typename T, int NT, bool kVec>
__device__ __forceinline__ void put8(T *row, int i, int t, int D, f32x8 x)
{
    if (kVec) {
        if (elem<NT, true>(i, 0, t) < D) store8(row + elem<NT, true>(i, 0, t), x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (elem<NT, false>(i, j, t) < D) row[elem<NT, false>(i, j, t)] = (T)x[j];
    }
}

// Such a piece as it lies in memory: half the registers for bf16 (backward with
// scale, 2^26 values, wide against as they lie: rows of 1024 271 and 225 us, 4096
// 236 and 195, 16384 403 and 245, 256 263 and 213, 5120 233 and 187, 8192 203 and
// 191; only where a row fills its threads and they had registers enough it loses,
// 512: 203 and 211, 2048: 174 and 182).  again() hides that the values have been
// widened before, or the compiler would keep them wide.
template <typename T, bool kVec>
struct Piece {
    f32x8 x;
    template <int NT>
    __device__ __forceinline__ void get(const T *row, int i, int t, int D) { x = get8<T, NT, kVec>(row, i, t, D); }
    __device__ __forceinline__ void clear() { x = zero8(); }
    __device__ __forceinline__ f32x8 wide() const { return x; }
    __device__ __forceinline__ void again() {}
};
template <>
struct Piece<bf16, true> {
    uint32_t u[4];
    template <int NT>
    __device__ __forceinline__ void get(const bf16 *row, int i, int t, int D)
    {
        clear();
        if (elem<NT, true>(i, 0, t) < D) __builtin_memcpy(u, row + elem<NT, true>(i, 0, t), 16);
    }
    __device__ __forceinline__ void clear() { u[0] = u[1] = u[2] = u[3] = 0; }
    __device__ __forceinline__ f32x8 wide() const
    {
        f32x8 x;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            x[2 * n] = bf16_lo(u[n]);
            x[2 * n + 1] = bf16_hi(u[n]);
        }
        return x;
    }
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int n = 0; n < 4; ++n) asm("" : "+v"(u[n]));
    }
};

// Sums of a and b over the row's NT threads.  `turn` alternates from call to
// call, so that one barrier per call is enough.
template <int NT>
__device__ __forceinline__ void row_sums(float &a, float &b, float (*red)[2][16], int turn)
{
    a = group_allreduce<16>(a);
    b = group_allreduce<16>(b);
    a += __shfl_xor(a, 16);
    b += __shfl_xor(b, 16);
    a += __shfl_xor(a, 32);
    b += __shfl_xor(b, 32);
    if (NT > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[turn][0][w] = a;
            red[turn][1][w] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            a += red[turn][0][i];
            b += red[turn][1][i];
        }
    }
}

template <typename T, int NT, int kN, bool kVec>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_fwd_kernel(NormArgs<T> a)
{
    constexpr int RB = NT < 256 ? 256 / NT : 1;   // rows per workgroup
    __shared__ float red[2][2][16];
    const int t = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * RB + threadIdx.x / NT;
    if (row >= a.rows) return;   // whole waves; with NT > 64, whole workgroups
    f32x8 x[kN];
    float ss = 0.f, none = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        x[i] = get8<T, NT, kVec>(a.x + row * a.D, i, t, a.D);
        if (a.y) {
            const f32x8 y = get8<T, NT, kVec>(a.y + row * a.D, i, t, a.D);
            x[i] += a.scale ? y * get8<float, NT, kVec>(a.scale, i, t, a.D) : y;
        }
        ss += sum8(x[i] * x[i]);
    }
    row_sums<NT>(ss, none, red, 0);
    const float r = 1.f / sqrtf(ss / a.D + a.eps);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if (a.xo) put8<T, NT, kVec>(a.xo + row * a.D, i, t, a.D, x[i]);
        put8<T, NT, kVec>(a.h + row * a.D, i, t, a.D, x[i] * r * get8<float, NT, kVec>(a.w, i, t, a.D));
    }
}

// Workgroup p: rows p * per ..; NT = 64 gives each of its waves every 4th.
template <typename T, int NT, int kN, bool kVec, bool kScale>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_bwd_kernel(NormArgs<T> a)
{
    constexpr int RB = NT < 256 ? 256 / NT : 1;
    __shared__ float red[2][2][16];
    // the longest rows read w and scale again for every row, from the cache:
    // 1024 threads have 128 registers each (4096 rows of 16384: bf16 245 -> 229
    // us, fp32 506 -> 449)
    constexpr bool kHold = !(NT == 1024 && kN == 2 && kScale);
    const int t = threadIdx.x % NT, grp = threadIdx.x / NT;
    f32x8 w[kN], sc[kN], dw[kN], ds[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if (kHold) w[i] = get8<float, NT, kVec>(a.w, i, t, a.D);
        if (kHold && kScale) sc[i] = get8<float, NT, kVec>(a.scale, i, t, a.D);
        dw[i] = ds[i] = zero8();
    }
    auto weight = [&](int i) { return kHold ? w[i] : get8<float, NT, kVec>(a.w, i, t, a.D); };
    const int64_t first = (int64_t)blockIdx.x * a.per;
    const int64_t end = first + a.per < a.rows ? first + a.per : a.rows;
    int turn = 0;
    for (int64_t row = first + grp; row < end; row += RB, turn ^= 1) {
        const int64_t o = row * a.D;
        Piece<T, kVec> xp[kN], hp[kN], dp[kN], yp[kN];
        float ss = 0.f, sm = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            xp[i].template get<NT>(a.x + o, i, t, a.D);
            hp[i].template get<NT>(a.dh + o, i, t, a.D);
            if (a.dxo)
                dp[i].template get<NT>(a.dxo + o, i, t, a.D);
            else
                dp[i].clear();
            if (kScale) yp[i].template get<NT>(a.y + o, i, t, a.D);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const f32x8 x = xp[i].wide();
            ss += sum8(x * x);
            sm += sum8(hp[i].wide() * weight(i) * x);
            xp[i].again();
            hp[i].again();
        }
        row_sums<NT>(ss, sm, red, turn);
        const float r = 1.f / sqrtf(ss / a.D + a.eps), m = sm / a.D * r;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const f32x8 xn = xp[i].wide() * r, dh = hp[i].wide();
            dw[i] += dh * xn;
            const f32x8 dx = dp[i].wide() + r * (dh * weight(i) - xn * m);
            put8<T, NT, kVec>(a.dx + o, i, t, a.D, dx);
            if (kScale) {
                put8<T, NT, kVec>(a.dy + o, i, t, a.D, dx * (kHold ? sc[i] : get8<float, NT, kVec>(a.scale, i, t, a.D)));
                ds[i] += dx * yp[i].wide();
            }
        }
    }
    float *part = a.part + ((int64_t)blockIdx.x * RB + grp) * (kScale ? 2 : 1) * a.D;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        put8<float, NT, kVec>(part, i, t, a.D, dw[i]);
        if (kScale) put8<float, NT, kVec>(part + a.D, i, t, a.D, ds[i]);
    }
}

template <typename T, int NT, int kN, bool kVec>
hipError_t norm_t(const NormLaunch &a, bool backward, hipStream_t stream)
{
    constexpr int RB = NT < 256 ? 256 / NT : 1, B = NT < 256 ? 256 : NT;
    NormArgs<T> p;
    p.x = static_cast<const T *>(backward ? a.x_out : a.x);
    p.y = static_cast<const T *>(a.y);
    p.dh = static_cast<const T *>(a.dh);
    p.dxo = static_cast<const T *>(a.dx_out);
    p.scale = a.scale;
    p.w = a.w;
    p.xo = static_cast<T *>(a.x_out);
    p.h = static_cast<T *>(a.h);
    p.dx = static_cast<T *>(a.dx);
    p.dy = static_cast<T *>(a.dy);
    p.part = a.part;
    p.rows = a.rows;
    p.D = (int)a.D;
    p.eps = a.eps;
    if (!backward) {
        const int64_t most = max_blocks(B) * RB;   // rows of a launch
        for (int64_t left = a.rows; left > 0; left -= most) {
            p.rows = left < most ? left : most;
            hipLaunchKernelGGL((norm_fwd_kernel<T, NT, kN, kVec>), dim3((unsigned)((p.rows + RB - 1) / RB)), dim3(B), 0,
                               stream, p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            p.x += most * a.D;
            p.h += most * a.D;
            if (p.y) p.y += most * a.D;
            if (p.xo) p.xo += most * a.D;
        }
        return hipSuccess;
    }
    const int64_t groups = norm_parts(a.rows, a.D) / RB;
    p.per = (a.rows + groups - 1) / groups;
    if (a.scale)
        hipLaunchKernelGGL((norm_bwd_kernel<T, NT, kN, kVec, true>), dim3((unsigned)groups), dim3(B), 0, stream, p);
    else
        hipLaunchKernelGGL((norm_bwd_kernel<T, NT, kN, kVec, false>), dim3((unsigned)groups), dim3(B), 0, stream, p);
    hipError_t e = hipGetLastError();
    const int64_t stride = a.scale ? 2 * a.D : a.D;
    for (int i = 0; i < (a.scale ? 2 : 1) && e == hipSuccess; ++i) {
        hipLaunchKernelGGL(parts_kernel, dim3((unsigned)((a.D + 63) / 64), 1), dim3(1024), 0, stream,
                           a.part + i * a.D, i ? a.dscale : a.dw, groups * RB, a.D, stride, (int64_t)0);
        e = hipGetLastError();
    }
    return e;
}

// Threads of a row: 64 up to D = 1024, 256 up to 4096, 1024 up to 16384
// (at most 16 values of each tensor per thread).
template <typename T, bool kVec>
hipError_t norm_d(const NormLaunch &a, bool backward, hipStream_t stream)
{
    if (a.D <= 512) return norm_t<T, 64, 1, kVec>(a, backward, stream);
    if (a.D <= 1024) return norm_t<T, 64, 2, kVec>(a, backward, stream);
    if (a.D <= 2048) return norm_t<T, 256, 1, kVec>(a, backward, stream);
    if (a.D <= 4096) return norm_t<T, 256, 2, kVec>(a, backward, stream);
    if (a.D <= 8192) return norm_t<T, 1024, 1, kVec>(a, backward, stream);
    return norm_t<T, 1024, 2, kVec>(a, backward, stream);
}

hipError_t norm_any(const NormLaunch &a, bool backward, hipStream_t stream)
{
    if (a.D % 8 == 0)   // rows of 8-value accesses are aligned
        return a.dtype == WKV7_F32 ? norm_d<float, true>(a, backward, stream) : norm_d<bf16, true>(a, backward, stream);
    return a.dtype == WKV7_F32 ? norm_d<float, false>(a, backward, stream) : norm_d<bf16, false>(a, backward, stream);
}

}  // namespace

int64_t epilogue_parts(int64_t rows, int64_t H, int64_t N, int64_t Hw)
{
    // about 2048 workgroups in all, each with at least a pass over its lanes
    const int64_t all = rows * H / Hw, R = 256 / (N / 8);
    int64_t p = (2048 + Hw - 1) / Hw;
    if (p > (all + R - 1) / R) p = (all + R - 1) / R;
    return p < 1 ? 1 : p;
}

int64_t norm_parts(int64_t rows, int64_t D)
{
    // about 1024 workgroups; with 64 threads to a row, four parts in each
    const int64_t RB = D <= 1024 ? 4 : 1;
    int64_t g = (rows + RB - 1) / RB;
    if (g > 1024) g = 1024;
    return (g < 1 ? 1 : g) * RB;
}

hipError_t launch_epilogue_forward(const EpilogueLaunch &a, hipStream_t stream)
{
    return a.dtype == WKV7_F32 ? epilogue_n<float>(a, false, stream) : epilogue_n<bf16>(a, false, stream);
}
hipError_t launch_epilogue_backward(const EpilogueLaunch &a, hipStream_t stream)
{
    return a.dtype == WKV7_F32 ? epilogue_n<float>(a, true, stream) : epilogue_n<bf16>(a, true, stream);
}
hipError_t launch_norm_forward(const NormLaunch &a, hipStream_t stream) { return norm_any(a, false, stream); }
hipError_t launch_norm_backward(const NormLaunch &a, hipStream_t stream) { return norm_any(a, true, stream); }

}  // namespace gdr
}  // namespace wkv7
