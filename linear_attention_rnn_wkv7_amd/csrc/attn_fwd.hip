// Causal softmax attention, forward.
//
// One pass over the keys with the running maximum m and sum l of each row:
//     s = c (q . k),  c = scale log2 e;   p = 2^(s - m);   l += p;   O += p v
// and y = O / l, lse = (m + log2 l) ln 2.  Where m has to change, l and O are
// multiplied by 2^(old - new); it need not be the maximum itself, and follows that
// only when p would pass 2^8.
//
// A workgroup of four waves has kTile rows of one head, 32 to a wave, which
// hold q (operand) and O^T (results) in registers; keys and values go by blocks
// through two buffers in LDS, the next copied while one is computed.  The narrow
// form, for few rows, has 32 of them, and each wave every fourth 32 keys.
//
// bf16 weights: one rounding of half a step before their product with v, as large as
// that of y.  In fp32 nothing is rounded on the way.
//
// Bound by matrix and vector instructions in turn: a 32 x 32 tile of heads of 64 is
// 256 cycles of the matrix unit and about 280 of the vector unit (16 exponentials of
// 8, the maximum, sum and conversion), of which three or four waves on a SIMD overlap
// most.  16384 tokens, 32 / 4 heads of 64: 1.13 to 1.18 ms, 930 to 970 TFLOP/s (a
// large product of matrices: 1300); 4 x 4096, 16 / 4 heads of 128: 283 us, 970; 24
// prompts of 12288 tokens, 32 / 8 heads of 128: 131 us, 530 (short rows: the fill and
// end of each workgroup).  fp32, 4096 tokens, 16 heads of 64: 400 us, 86 TFLOP/s
// (153).  Slower or equal: 64 rows to a wave, scores of a block ahead, three or four
// buffers.

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
    uint32_t chunk;
    float scale;
};

// Keys of a block.  With wide heads in bf16, 32 of them make room for a third
// workgroup on the compute unit, which pays where the rows are short: 12288 tokens
// in 24 prompts, 32 / 8 heads of 128, 137 us with 64 and 128 with 32; 4 x 4096 x 16 /
// 4 290 and 279.  Heads of 64 (four workgroups either way) 666 and 714 (8 x 4096 x 32).
template <typename T, int D>
constexpr int kKeysOf = sizeof(T) == 2 && D == 128 ? 32 : 64;

// 32 rows of a wave.
template <typename T, int D>
struct Rows {
    Tile<T, D> tl;
    Oct<T> q[D / 16];
    f32x16 o[D / 32];
    float ref, l, c;   // ref: what stands for the maximum, times c
    int row0, row, half;

    __device__ __forceinline__ void init(const FwdArgs<T> &p, const Place &at, int h, int first, int lane)
    {
        tl.init(lane);
        half = lane >> 5;
        row0 = first;
        row = row0 + (lane & 31);
        const int r = row < at.len ? row : at.len - 1;
        const T *qp = p.q + (at.tok + r) * p.q_stride + h * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) q[ks] = *reinterpret_cast<const Oct<T> *>(qp + 16 * ks);
        c = p.scale * kLog2e;
        clear();
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();
        ref = kLowest;
        l = 0.f;
    }
    // 32 N keys from key0 on; kMask where some row does not see all: the tile that begins
    // with the wave's first row is cut through, and what follows it hidden.
    template <int N, bool kMask, bool kCareful>
    __device__ __forceinline__ void keys(const char *kt, const char *vt, int key0)
    {
        using L = Tile<T, D>;
        f32x16 s[N];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            s[t] = zero16();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) s[t] = mma(tl.row(kt + L::bytes(32) * t, ks), q[ks], s[t]);
        }
        if constexpr (kMask) {
#pragma unroll
            for (int t = 0; t < N; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * t + reg_row(i, half) > row) s[t][i] = kNegInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < N; ++t)
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
        float sum[N];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            sum[t] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -ref));
                sum[t] += s[t][i];
            }
#pragma unroll
            for (int ss = 0; ss < 2; ++ss) {
                const Oct<T> w = as_operand<T>(s[t], ss);
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) {
                    Oct<T> x = tl.col(vt, dt, 2 * t + ss);
                    if (kCareful && kMask && key0 + 32 * t >= row0) x = finite_of<T>(x);
                    o[dt] = mma(x, w, o[dt]);
                }
            }
            l += sum[t];
        }
    }
    // After the last of them, with care: what was left out of the tile that is cut through.
    __device__ __forceinline__ void finish(const T *vp, int64_t stride, int len)
    {
        int own = row;
        asm volatile("" : "+v"(own));   // else a register holds row - row0 from the start
        add_odd<T, D, false>(o, vp + row0 * stride, stride, len - row0 < 32 ? len - row0 : 32, (2u << (own - row0)) - 1,
                             half);
    }
};

// Four values of y at entry e, and what their rounding takes away.
template <typename T>
__device__ __forceinline__ void store_y(const FwdArgs<T> &p, int64_t e, f32x4 x)
{
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

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? (D == 64 ? 4 : 3) : 1) attn_fwd_kernel(FwdArgs<T> p)
{
    constexpr int kKeys = kKeysOf<T, D>, kBytes = Tile<T, D>::bytes(kKeys);
    __shared__ __attribute__((aligned(16))) char lds[2][2][kBytes];   // [buffer][k, v]
    __shared__ int finite[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, h;
    unit_of(p.seqs, p.B, p.Hq, p.chunk, true, blockIdx.x, slot, h);
    const Place at = locate<kTile>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int hk = h / p.group;
    const T *kp = uniform(p.k + at.tok * p.k_stride + hk * D), *vp = uniform(p.v + at.tok * p.v_stride + hk * D);

    const int end = at.at + kTile < at.len ? at.at + kTile : at.len;   // keys that any row sees
    const int blocks = (end + kKeys - 1) / kKeys;
    Copy<T, D, kKeys, 4> ck, cv;
    ck.init(p.k_stride, wave, lane);
    cv.init(p.v_stride, wave, lane);
    const unsigned base = lds_address(lds);
    auto first = [&]() __attribute__((always_inline)) {
        ck.issue(base, kp, at.len, wave, lane);
        cv.issue(base + kBytes, vp, at.len, wave, lane);
    };
    first();
    const int row0 = at.at + 32 * wave;
    Rows<T, D> r;
    r.init(p, at, h, row0, lane);
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
    auto pass = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(careful)::value;
        int n = 0;
        for (; n < at.at / kKeys; ++n) {   // every row sees all of these
            const auto *kv = arrive(n);
            r.template keys<kKeys / 32, false, kCareful>(kv[0], kv[1], n * kKeys);
        }
        for (; n < blocks; ++n) {
            const auto *kv = arrive(n);
            if (n * kKeys <= row0 + 31 && row0 < at.len)
                r.template keys<kKeys / 32, true, kCareful>(kv[0], kv[1], n * kKeys);
        }
    };
    pass(std::false_type{});
    if (!all_waves(all_finite(r.o), finite, wave, lane)) {
        first();
        r.clear();
        pass(std::true_type{});
        if (row0 < at.len) r.finish(vp, p.v_stride, at.len);
    }
    if (r.row >= at.len) return;
    const float l = half_sum(r.l), inv = 1.f / l;
    const int64_t to = (at.tok + r.row) * p.Hq + h;
    if (p.lse && r.half == 0) p.lse[to] = (r.ref + __builtin_amdgcn_logf(l)) * kLn2;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            store_y(p, to * D + 32 * dt + reg_row(i, r.half),
                    f32x4{r.o[dt][i], r.o[dt][i + 1], r.o[dt][i + 2], r.o[dt][i + 3]} * inv);
}

template <typename T, int D>
__global__ void __launch_bounds__(256, 1) attn_fwd_narrow_kernel(FwdArgs<T> p)
{
    using O = Own<T, D>;
    __shared__ __attribute__((aligned(16))) char lds[4][O::kWave];
    __shared__ float stat[4][2][kNarrow];   // reference, sum
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, h;
    unit_of(p.seqs, p.B, p.Hq, p.chunk, true, blockIdx.x, slot, h);
    const Place at = locate<kNarrow>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int hk = h / p.group;
    const T *kp = uniform(p.k + at.tok * p.k_stride + hk * D), *vp = uniform(p.v + at.tok * p.v_stride + hk * D);
    Copy<T, D, 32, 1> ck, cv;
    ck.init(p.k_stride, 0, lane);
    cv.init(p.v_stride, 0, lane);
    const unsigned base = lds_address(lds[wave]);
    const int last = at.at / 32;   // 32 keys to a step, the last of them masked
    auto send = [&](int n) __attribute__((always_inline)) {
        const unsigned to = base + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
        const int64_t first = (int64_t)n * 32;
        ck.issue(to, kp + first * p.k_stride, at.len - (int)first, 0, lane);
        cv.issue(to + O::kBytes, vp + first * p.v_stride, at.len - (int)first, 0, lane);
    };
    if (wave <= last) send(wave);
    Rows<T, D> r;
    r.init(p, at, h, at.at, lane);
    auto pass = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(careful)::value;
        for (int n = wave; n <= last; n += 4) {
            wait_dma();
            if (O::kBuffers == 2 && n + 4 <= last) send(n + 4);
            const char *kv = lds[wave] + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
            if (n < last)
                r.template keys<1, false, kCareful>(kv, kv + O::kBytes, n * 32);
            else
                r.template keys<1, true, kCareful>(kv, kv + O::kBytes, n * 32);
            reads_done();
            if (O::kBuffers == 1 && n + 4 <= last) send(n + 4);
        }
    };
    pass(std::false_type{});
    if (!all_finite(r.o)) {   // (a wave by itself)
        send(wave);
        r.clear();
        pass(std::true_type{});
        if (last % 4 == wave) r.finish(vp, p.v_stride, at.len);
    }
    r.l = half_sum(r.l);
    if (r.half == 0) {
        stat[wave][0][lane] = r.ref;
        stat[wave][1][lane] = r.l;
    }
    put_rows<D>(lds[wave], r.o, lane);
    __syncthreads();
    constexpr int kLanes = D / 4;
    for (int i = threadIdx.x / kLanes; i < kNarrow && at.at + i < at.len; i += 256 / kLanes) {
        const int col = 4 * (threadIdx.x % kLanes);
        float top = kLowest, l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[w][0][i]);
        f32x4 x = gdr::zero4();
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float a = __builtin_amdgcn_exp2f(stat[w][0][i] - top);
            l += a * stat[w][1][i];
            x += a * get_row<D>(lds[w], i, col);
        }
        const int64_t to = (at.tok + at.at + i) * p.Hq + h;
        if (p.lse && col == 0) p.lse[to] = (top + __builtin_amdgcn_logf(l)) * kLn2;
        store_y(p, to * D + col, x * (1.f / l));
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
    p.chunk = chunk_of(a.seqs, a.seqs.starts ? a.Hq : a.B * a.Hq, a.seqs.T * 2 * D * (int64_t)sizeof(T), p.group);
    if (is_narrow(a.seqs.slots * a.Hq, a.dtype)) {
        p.seqs = narrow(a.seqs, a.B);
        hipLaunchKernelGGL((attn_fwd_narrow_kernel<T, D>), dim3((unsigned)(p.seqs.slots * a.Hq)), dim3(256), 0, stream,
                           p);
    } else {
        hipLaunchKernelGGL((attn_fwd_kernel<T, D>), dim3((unsigned)(a.seqs.slots * a.Hq)), dim3(256), 0, stream, p);
    }
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
