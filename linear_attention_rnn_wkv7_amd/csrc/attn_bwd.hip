// Causal softmax attention, gradients.
//
// With P_ij = exp(s_ij - lse_i) and D_i = dy_i . y_i:
//     dv_j = sum_i P_ij dy_i,   dS_ij = P_ij (dy_i . v_j - D_i)
//     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i
// P is formed again from q, k and lse.  Three kernels: D and lse log2 e of
// every token and head into a table; dk and dv, a workgroup to kTile keys,
// which goes over the queries behind them, of every query head that reads the
// key head, in order; dq, a workgroup to kTile queries, which goes over the keys
// before them.  The scores and dy . v are formed twice (7 products instead of
// 5): dq would otherwise be a sum over workgroups, by atomics in an order of
// their own.

#include <type_traits>

#include "attn_device.h"

namespace wkv7 {
namespace attn {
namespace {

template <typename T>
struct BwdArgs {
    Seqs seqs;
    const T *q, *k, *v, *y, *dy;
    const float *lse;
    const bf16 *record;
    T *dq, *dk, *dv;
    f32x2 *stats;   // [Hq][tokens]: lse log2 e, D
    int64_t B, Hq, Hk, q_stride, k_stride, v_stride, tokens;
    int group;
    float scale;
};

template <typename T>
__device__ __forceinline__ f32x8 wide(Oct<T> x)
{
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __builtin_convertvector(x, f32x8);
}

// D / 8 lanes to a token's head, heads side by side.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_stats_kernel(BwdArgs<T> p)
{
    constexpr int L = D / 8;
    const int64_t all = p.tokens * p.Hq;
    for (int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; row < all;   // whole rows
         row += (int64_t)gridDim.x * (256 / L)) {
        const int64_t e = row * D + 8 * (threadIdx.x % L);
        const f32x8 dy = wide<T>(*reinterpret_cast<const Oct<T> *>(p.dy + e));
        f32x8 y = wide<T>(*reinterpret_cast<const Oct<T> *>(p.y + e));
        if (sizeof(T) == 2 && p.record) y += wide<bf16>(*reinterpret_cast<const bf16x8 *>(p.record + e));
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(dy[j], y[j], d);
        d = group_allreduce<L>(d);
        if (threadIdx.x % L == 0) {
            const int64_t tok = row / p.Hq, h = row - tok * p.Hq;
            p.stats[h * p.tokens + tok] = f32x2{p.lse[row] * kLog2e, d};
        }
    }
}

constexpr int kRows = 64;   // of q and dy, or of k and v, in LDS at a time

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 && D == 64 ? 2 : 1) attn_dkdv_kernel(BwdArgs<T> p)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(kRows);
    __shared__ __attribute__((aligned(16))) char lds[2][2][kBytes];   // [buffer][q, dy]
    __shared__ __attribute__((aligned(16))) float table[2][2][kRows];   // [buffer][lse, D]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, l32 = lane & 31;
    L tl;
    tl.init(lane);
    int64_t slot, hk;
    unit_of(p.seqs, p.B, p.Hk, false, blockIdx.x, slot, hk);
    const Place at = locate(p.seqs, slot);
    if (at.len == 0) return;
    const int key0 = at.at + 32 * wave, key = key0 + l32;
    Oct<T> k[D / 16], v[D / 16];
    {
        const int64_t r = at.tok + (key < at.len ? key : at.len - 1);
        const T *kp = p.k + r * p.k_stride + hk * D + 8 * half, *vp = p.v + r * p.v_stride + hk * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            k[ks] = *reinterpret_cast<const Oct<T> *>(kp + 16 * ks);
            v[ks] = *reinterpret_cast<const Oct<T> *>(vp + 16 * ks);
        }
    }
    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) dk[dt] = dv[dt] = zero16();
    const float c = p.scale * kLog2e;

    // 32 rows of queries for the wave's keys; kMask where some see not all of them.
    auto rows = [&](const char *qt, const char *yt, const float *lses, const float *ds_, int r0, auto mask)
                    __attribute__((always_inline)) {
        constexpr bool kMask = decltype(mask)::value;
        f32x16 s = zero16(), ds = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) s = mma(tl.row(qt, ks), k[ks], s);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) ds = mma(tl.row(yt, ks), v[ks], ds);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 lse = *reinterpret_cast<const f32x4 *>(lses + reg_row(i, half));
            const f32x4 dd = *reinterpret_cast<const f32x4 *>(ds_ + reg_row(i, half));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = __builtin_amdgcn_exp2f(fmaf(s[i + j], c, -lse[j]));
                s[i + j] = w;
                ds[i + j] = w * (ds[i + j] - dd[j]);
            }
        }
        if constexpr (kMask) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = r0 + reg_row(i, half);
                if (r < key) s[i] = ds[i] = 0.f;
            }
        }
#pragma unroll
        for (int ss = 0; ss < 2; ++ss) {
            const Oct<T> w = as_operand<T>(s, ss), dw = as_operand<T>(ds, ss);
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) {
                dv[dt] = mma(tl.col(yt, dt, ss), w, dv[dt]);
                dk[dt] = mma(tl.col(qt, dt, ss), dw, dk[dt]);
            }
        }
    };

    const int first = at.at / kRows, last = (at.len + kRows - 1) / kRows;
    const int64_t h_end = (hk + 1) * p.group;
    Copy<T, D, kRows, 4> cq, cy;
    cq.init(p.q_stride, wave, lane);
    cy.init(p.Hq * D, wave, lane);
    const unsigned base = lds_address(lds);
    f32x2 ahead;
    auto issue = [&](int buffer, int64_t h, int block) __attribute__((always_inline)) {
        const int row0 = block * kRows, rows = at.len - row0;
        cq.issue(base + buffer * 2 * kBytes, p.q + (at.tok + row0) * p.q_stride + h * D, rows, wave, lane);
        cy.issue(base + buffer * 2 * kBytes + kBytes, p.dy + ((at.tok + row0) * p.Hq + h) * D, rows, wave, lane);
        if (wave == 0) {   // rows that are not there have no weights
            ahead = f32x2{-kNegInf, 0.f};
            if (lane < rows) ahead = p.stats[h * p.tokens + at.tok + row0 + lane];
        }
    };
    // Waits for block `block` of head h and sends for the next one.
    int buffer = 1;
    auto arrive = [&](int64_t h, int block) __attribute__((always_inline)) {
        buffer ^= 1;
        wait_dma();
        if (wave == 0) {
            table[buffer][0][lane] = ahead[0];
            table[buffer][1][lane] = ahead[1];
        }
        __syncthreads();
        if (block + 1 < last)
            issue(buffer ^ 1, h, block + 1);
        else if (h + 1 < h_end)
            issue(buffer ^ 1, h + 1, first);
    };
    issue(0, hk * p.group, first);
    for (int64_t h = hk * p.group; h < h_end; ++h) {
        int block = first;
        for (; block < last && block < first + kTile / kRows; ++block) {
            arrive(h, block);
            for (int t = 0; t < 2; ++t)
                if (block * kRows + 32 * t + 31 >= key0 && key0 < at.len)
                    rows(lds[buffer][0] + L::bytes(32) * t, lds[buffer][1] + L::bytes(32) * t,
                         &table[buffer][0][32 * t], &table[buffer][1][32 * t], block * kRows + 32 * t, std::true_type{});
        }
        for (; block < last; ++block) {   // these rows see every key
            arrive(h, block);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                rows(lds[buffer][0] + L::bytes(32) * t, lds[buffer][1] + L::bytes(32) * t,
                     &table[buffer][0][32 * t], &table[buffer][1][32 * t], block * kRows + 32 * t, std::false_type{});
        }
    }
    if (key >= at.len) return;
    const int64_t to = ((at.tok + key) * p.Hk + hk) * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int64_t e = to + 32 * dt + reg_row(i, half);
            const f32x4 a = f32x4{dk[dt][i], dk[dt][i + 1], dk[dt][i + 2], dk[dt][i + 3]} * p.scale;
            const f32x4 b = f32x4{dv[dt][i], dv[dt][i + 1], dv[dt][i + 2], dv[dt][i + 3]};
            *reinterpret_cast<Quad<T> *>(p.dk + e) = __builtin_convertvector(a, Quad<T>);
            *reinterpret_cast<Quad<T> *>(p.dv + e) = __builtin_convertvector(b, Quad<T>);
        }
}

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) attn_dq_kernel(BwdArgs<T> p)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(kRows);
    __shared__ __attribute__((aligned(16))) char lds[2][2][kBytes];   // [buffer][k, v]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, l32 = lane & 31;
    L tl;
    tl.init(lane);
    int64_t slot, h;
    unit_of(p.seqs, p.B, p.Hq, true, blockIdx.x, slot, h);
    const Place at = locate(p.seqs, slot);
    if (at.len == 0) return;
    const int64_t hk = h / p.group;
    const T *kp = p.k + at.tok * p.k_stride + hk * D, *vp = p.v + at.tok * p.v_stride + hk * D;
    const int row0 = at.at + 32 * wave, row = row0 + l32;
    Oct<T> q[D / 16], dy[D / 16];
    f32x2 st;
    {
        const int64_t r = at.tok + (row < at.len ? row : at.len - 1);
        const T *qp = p.q + r * p.q_stride + h * D + 8 * half, *yp = p.dy + (r * p.Hq + h) * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            q[ks] = *reinterpret_cast<const Oct<T> *>(qp + 16 * ks);
            dy[ks] = *reinterpret_cast<const Oct<T> *>(yp + 16 * ks);
        }
        st = p.stats[h * p.tokens + r];
    }
    f32x16 dq[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) dq[dt] = zero16();
    const float c = p.scale * kLog2e;
    // 32 keys for the wave's rows; kMask where some row does not see all of them.
    auto keys = [&](const char *kt, const char *vt, int key0, auto mask) __attribute__((always_inline)) {
        constexpr bool kMask = decltype(mask)::value;
        f32x16 s = zero16(), ds = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) s = mma(tl.row(kt, ks), q[ks], s);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) ds = mma(tl.row(vt, ks), dy[ks], ds);
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -st[0])) * (ds[i] - st[1]);
        if constexpr (kMask) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (key0 + reg_row(i, half) > row) ds[i] = 0.f;
        }
#pragma unroll
        for (int ss = 0; ss < 2; ++ss) {
            const Oct<T> w = as_operand<T>(ds, ss);
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) dq[dt] = mma(tl.col(kt, dt, ss), w, dq[dt]);
        }
    };

    const int end = at.at + kTile < at.len ? at.at + kTile : at.len;
    const int blocks = (end + kRows - 1) / kRows;
    Copy<T, D, kRows, 4> ck, cv;
    ck.init(p.k_stride, wave, lane);
    cv.init(p.v_stride, wave, lane);
    const unsigned base = lds_address(lds);
    ck.issue(base, kp, at.len, wave, lane);
    cv.issue(base + kBytes, vp, at.len, wave, lane);
    auto arrive = [&](int n) __attribute__((always_inline)) {
        wait_dma();
        __syncthreads();
        if (n + 1 < blocks) {
            const unsigned to = base + ((n + 1) & 1) * 2 * kBytes;
            const int64_t next = (int64_t)(n + 1) * kRows;
            ck.issue(to, kp + next * p.k_stride, at.len - (int)next, wave, lane);
            cv.issue(to + kBytes, vp + next * p.v_stride, at.len - (int)next, wave, lane);
        }
        return lds[n & 1];
    };
    int n = 0;
    for (; n < at.at / kRows; ++n) {   // every row sees all of these
        const auto *kv = arrive(n);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            keys(kv[0] + L::bytes(32) * t, kv[1] + L::bytes(32) * t, n * kRows + 32 * t, std::false_type{});
    }
    for (; n < blocks; ++n) {
        const auto *kv = arrive(n);
        for (int t = 0; t < 2; ++t)
            if (n * kRows + 32 * t <= row0 + 31 && row0 < at.len)
                keys(kv[0] + L::bytes(32) * t, kv[1] + L::bytes(32) * t, n * kRows + 32 * t, std::true_type{});
    }
    if (row >= at.len) return;
    const int64_t to = ((at.tok + row) * p.Hq + h) * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 x = f32x4{dq[dt][i], dq[dt][i + 1], dq[dt][i + 2], dq[dt][i + 3]} * p.scale;
            *reinterpret_cast<Quad<T> *>(p.dq + to + 32 * dt + reg_row(i, half)) = __builtin_convertvector(x, Quad<T>);
        }
}

template <typename T, int D>
hipError_t launch_t(const Launch &a, hipStream_t stream)
{
    BwdArgs<T> p;
    p.seqs = a.seqs;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.v = static_cast<const T *>(a.v);
    p.y = static_cast<const T *>(a.y);
    p.dy = static_cast<const T *>(a.dy);
    p.lse = a.lse;
    p.record = static_cast<const bf16 *>(a.record);
    p.dq = static_cast<T *>(a.dq);
    p.dk = static_cast<T *>(a.dk);
    p.dv = static_cast<T *>(a.dv);
    p.stats = reinterpret_cast<f32x2 *>(a.stats);
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.tokens = a.B * a.seqs.T;
    p.group = (int)(a.Hq / a.Hk);
    p.scale = a.scale;
    const int64_t per = 256 / (D / 8);
    hipLaunchKernelGGL((attn_stats_kernel<T, D>), dim3(grid_of((p.tokens * a.Hq + per - 1) / per)), dim3(256), 0,
                       stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_dkdv_kernel<T, D>), dim3((unsigned)(a.seqs.slots * a.Hk)), dim3(256), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_dq_kernel<T, D>), dim3((unsigned)(a.seqs.slots * a.Hq)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_backward(const Launch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.D == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    return a.D == 64 ? launch_t<bf16, 64>(a, stream) : launch_t<bf16, 128>(a, stream);
}

}  // namespace attn
}  // namespace wkv7
