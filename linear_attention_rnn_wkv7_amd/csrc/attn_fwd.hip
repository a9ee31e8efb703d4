// Causal softmax attention, forward.
//
// One pass over the keys with the running maximum m and sum l of each row:
//     s = c (q . k),  c = scale log2 e;   p = 2^(s - m);   l += p;   O += p v
// and y = O / l, lse = (m + log2 l) ln 2.  Where m has to change, l and O are
// multiplied by 2^(old - new); it need not be the maximum itself, and follows that
// only when p would pass 2^8.
//
// A workgroup of four waves has kTile rows of one head, 32 to a wave, which
// hold q (operand) and O^T (results) in registers; keys and values go by 64
// through two buffers in LDS, the next copied while one is computed.

#include <type_traits>

#include "attn_device.h"

namespace wkv7 {
namespace attn {
namespace {

template <typename T>
struct FwdArgs {
    Seqs seqs;
    const T *q, *k, *v;
    T *y;
    float *lse;
    bf16 *record;
    int64_t B, Hq, Hk, q_stride, k_stride, v_stride;
    int group;
    float scale;
};

constexpr int kKeys = 64;

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) attn_fwd_kernel(FwdArgs<T> p)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(kKeys);
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
    Oct<T> q[D / 16];
    {
        const int r = row < at.len ? row : at.len - 1;
        const T *qp = p.q + (at.tok + r) * p.q_stride + h * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) q[ks] = *reinterpret_cast<const Oct<T> *>(qp + 16 * ks);
    }
    f32x16 o[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();
    float ref = kNegInf, l = 0.f;   // ref: the maximum times c
    const float c = p.scale * kLog2e;

    // One block of keys for the wave's rows; kMask where some row does not see all.
    auto block = [&](const char *kt, const char *vt, int key0, auto mask) __attribute__((always_inline)) {
        constexpr bool kMask = decltype(mask)::value;
        f32x16 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = zero16();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) s[t] = mma(tl.row(kt + L::bytes(32) * t, ks), q[ks], s[t]);
        }
        if constexpr (kMask) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * t + reg_row(i, half) > row) s[t][i] = kNegInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = half_max(top) * c;
        // a row keeps its reference until its maximum is 2^8 times what that stands for
        const bool grown = top > ref + 8.f;
        if (__any(grown)) {
            const float to = grown ? top : ref, alpha = __builtin_amdgcn_exp2f(grown ? ref - to : 0.f);
            ref = to;
            l *= alpha;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= alpha;
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -ref));
                sum[t] += s[t][i];
            }
#pragma unroll
            for (int ss = 0; ss < 2; ++ss) {
                const Oct<T> w = as_operand<T>(s[t], ss);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) o[dt] = mma(tl.col(vt, dt, 2 * t + ss), w, o[dt]);
            }
        }
        l += sum[0] + sum[1];
    };

    const int end = at.at + kTile < at.len ? at.at + kTile : at.len;   // keys that any row sees
    const int blocks = (end + kKeys - 1) / kKeys;
    Copy<T, D, kKeys, 4> ck, cv;
    ck.init(p.k_stride, wave, lane);
    cv.init(p.v_stride, wave, lane);
    const unsigned base = lds_address(lds);
    ck.issue(base, kp, at.len, wave, lane);
    cv.issue(base + kBytes, vp, at.len, wave, lane);
    // Waits for block n, sends for the next one, and gives block n's place.
    auto arrive = [&](int n) __attribute__((always_inline)) {
        wait_dma();
        __syncthreads();
        if (n + 1 < blocks) {
            const unsigned to = base + ((n + 1) & 1) * 2 * kBytes;
            const int64_t next = (int64_t)(n + 1) * kKeys;
            ck.issue(to, kp + next * p.k_stride, at.len - (int)next, wave, lane);
            cv.issue(to + kBytes, vp + next * p.v_stride, at.len - (int)next, wave, lane);
        }
        return lds[n & 1];
    };
    int n = 0;
    for (; n < at.at / kKeys; ++n) {   // every row sees all of these
        const auto *kv = arrive(n);
        block(kv[0], kv[1], n * kKeys, std::false_type{});
    }
    for (; n < blocks; ++n) {
        const auto *kv = arrive(n);
        if (n * kKeys <= row0 + 31 && row0 < at.len) block(kv[0], kv[1], n * kKeys, std::true_type{});
    }
    if (row >= at.len) return;
    l = half_sum(l);
    const float inv = 1.f / l;
    const int64_t to = (at.tok + row) * p.Hq + h;
    if (p.lse && half == 0) p.lse[to] = (ref + __builtin_amdgcn_logf(l)) * kLn2;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 x = f32x4{o[dt][i], o[dt][i + 1], o[dt][i + 2], o[dt][i + 3]} * inv;
            const int64_t e = to * D + 32 * dt + reg_row(i, half);
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<f32x4 *>(p.y + e) = x;
            } else {
                const bf16x4 r = __builtin_convertvector(x, bf16x4);
                *reinterpret_cast<bf16x4 *>(p.y + e) = r;
                if (p.record)
                    *reinterpret_cast<bf16x4 *>(p.record + e) =
                        __builtin_convertvector(x - __builtin_convertvector(r, f32x4), bf16x4);
            }
        }
}

template <typename T, int D>
hipError_t launch_t(const Launch &a, hipStream_t stream)
{
    FwdArgs<T> p;
    p.seqs = a.seqs;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.v = static_cast<const T *>(a.v);
    p.y = static_cast<T *>(a.y);
    p.lse = a.lse;
    p.record = static_cast<bf16 *>(a.record);
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.group = (int)(a.Hq / a.Hk);
    p.scale = a.scale;
    hipLaunchKernelGGL((attn_fwd_kernel<T, D>), dim3((unsigned)(a.seqs.slots * a.Hq)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_forward(const Launch &a, hipStream_t stream)
{
    if (a.dtype == WKV7_F32) return a.D == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    return a.D == 64 ? launch_t<bf16, 64>(a, stream) : launch_t<bf16, 128>(a, stream);
}

}  // namespace attn
}  // namespace wkv7
