// Causal softmax attention, gradients.
//
// With P_ij = exp(s_ij - lse_i) and D_i = dy_i . y_i:
//     dv_j = sum_i P_ij dy_i,   dS_ij = P_ij (dy_i . v_j - D_i)
//     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i
// P is formed again from q, k and lse.  Two kernels: dq, a workgroup to kTile
// queries, which goes over the keys before them, and which leaves D and lse log2 e
// of every token and head in a table; dk and dv, a workgroup to kTile keys, which
// goes over the queries behind them, of every query head that reads the key head,
// in order; narrow forms of both for few of them.  The scores and dy . v are
// formed twice (7 products instead of 5): dq would otherwise be a sum over
// workgroups, by atomics in an order of their own.
//
// bf16: P and dS are rounded once, by half a step, before their products with dy, q
// and k, as large as the outputs' own rounding.  D takes y with the record of what
// its rounding took away.
//
// Bound as the forward by matrix and vector instructions in turn, and at D = 128 by
// registers: with k, v, dk and dv of 32 keys a wave has a SIMD to itself.  8 x 4096,
// 32 heads of 64: dk and dv 1040 to 1070 us, dq 810, the matrix units busy 0.55 of the
// time; 4 x 4096, 16 / 4 heads of 128: 665 to 695 (busy 0.33) and 382.  Both together, 24
// sequences in 12288 tokens, 32 / 8 heads of 128: 574 us, 300 TFLOP/s of 5 products;
// fp32, 4096 tokens, 16 heads of 64: 1174 us, 73.  Slower for dk and dv: 64
// keys to a wave (heads of 64) 1726 against 1194; two waves with spills (128) 1177
// against 697, with v in LDS 1089 against 685; dk and dv apart 702 against 749 for the
// kernel, the same for a run of calls, in which the clock falls with more products.

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
    uint32_t chunk_q, chunk_k;   // units of a die at a time, of queries and of keys
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

constexpr int kRows = 64;   // of q and dy, or of k and v, in LDS at a time

// 32 keys of a wave.
template <typename T, int D>
struct Keys {
    Tile<T, D> tl;
    Oct<T> k[D / 16], v[D / 16];
    f32x16 dk[D / 32], dv[D / 32];
    float c;
    int key0, key, half;

    __device__ __forceinline__ void init(const BwdArgs<T> &p, const Place &at, int hk, int first, int lane)
    {
        tl.init(lane);
        half = lane >> 5;
        key0 = first;
        key = key0 + (lane & 31);
        const int64_t r = at.tok + (key < at.len ? key : at.len - 1);
        const T *kp = p.k + r * p.k_stride + hk * D + 8 * half, *vp = p.v + r * p.v_stride + hk * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            k[ks] = *reinterpret_cast<const Oct<T> *>(kp + 16 * ks);
            v[ks] = *reinterpret_cast<const Oct<T> *>(vp + 16 * ks);
        }
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) dk[dt] = dv[dt] = zero16();
        c = p.scale * kLog2e;
    }
    // 32 rows of queries from r0 on (len: the sequence's), with their table of lse and D;
    // kMask where some may not see all keys: the tile that begins with the wave's first
    // key is cut through.
    template <bool kMask, bool kCareful>
    __device__ __forceinline__ void rows(const char *qt, const char *yt, const float *lses, const float *dots, int r0,
                                         int len)
    {
        f32x16 s = zero16(), ds = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) s = mma(tl.row(qt, ks), k[ks], s);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) ds = mma(tl.row(yt, ks), v[ks], ds);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 lse = *reinterpret_cast<const f32x4 *>(lses + reg_row(i, half));
            const f32x4 dot = *reinterpret_cast<const f32x4 *>(dots + reg_row(i, half));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = __builtin_amdgcn_exp2f(fmaf(s[i + j], c, -lse[j]));
                s[i + j] = w;
                ds[i + j] = w * (ds[i + j] - dot[j]);
            }
        }
        if constexpr (kMask) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (r0 + reg_row(i, half) < key || (kCareful && r0 + reg_row(i, half) >= len)) s[i] = ds[i] = 0.f;
        }
#pragma unroll
        for (int ss = 0; ss < 2; ++ss) {
            const Oct<T> w = as_operand<T>(s, ss), dw = as_operand<T>(ds, ss);
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) {
                Oct<T> y = tl.col(yt, dt, ss);
                if (kCareful && r0 == key0) y = finite_of<T>(y);
                dv[dt] = mma(y, w, dv[dt]);
                Oct<T> q = tl.col(qt, dt, ss);
                if (kCareful && r0 == key0) q = finite_of<T>(q);
                dk[dt] = mma(q, dw, dk[dt]);
            }
        }
    }
    __device__ __forceinline__ void store(const BwdArgs<T> &p, const Place &at, int hk) const
    {
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
    // After the last of them, with care: what was left out of the tiles that are cut
    // through, of all the heads.  (A q that is not finite makes its scores, and so the
    // row's sum or its own weights.)
    __device__ __forceinline__ void finish(const BwdArgs<T> &p, const Place &at, int hk)
    {
        const int count = at.len - key0 < 32 ? at.len - key0 : 32;
        const int64_t first = at.tok + key0;
        for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
            add_odd<T, D, false>(dv, p.dy + (first * p.Hq + h) * D, p.Hq * D, count, ~0u << (key - key0), half);
            add_odd<T, D, true>(dk, p.q + first * p.q_stride + h * D, p.q_stride, count, ~0u << (key - key0), half);
        }
    }
};

// 32 keys by a wave, with care: after the forms below, where these have found results
// that are not finite.  Its tiles are in `lds`, the wave's own.  It makes all that it needs
// anew and stores its results itself: with anything shared between it and the loops of
// those forms, registers of these were kept in memory (heads of 64: up to 68 bytes, two
// reads of them between the copies of a step).
template <typename T, int D>
__device__ __forceinline__ void careful_keys(const BwdArgs<T> &p, Place at, int hk, int key0, char *lds, float *table)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(32);
    Keys<T, D> w;
    w.init(p, at, hk, key0, lane_anew());
#pragma unroll 1
    for (int h = hk * p.group; h < (hk + 1) * p.group; ++h)
#pragma unroll 1
        for (int row0 = key0; row0 < at.len; row0 += 32) {
            const int lane = lane_anew();
            Copy<T, D, 32, 1> cq, cy;
            cq.init(p.q_stride, 0, lane);
            cy.init(p.Hq * D, 0, lane);
            const int rows = at.len - row0;   // the others are zeros, with no weights
            cq.issue(lds_address(lds), p.q + (at.tok + row0) * p.q_stride + h * D, rows, 0, lane);
            cy.issue(lds_address(lds) + kBytes, p.dy + ((at.tok + row0) * p.Hq + h) * D, rows, 0, lane);
            f32x2 st = {-kNegInf, 0.f};
            if ((lane & 31) < rows) st = p.stats[h * p.tokens + at.tok + row0 + (lane & 31)];
            wait_dma();
            cq.clear(lds, rows, 0, lane);
            cy.clear(lds + kBytes, rows, 0, lane);
            table[lane] = st[lane >> 5];
            gdr::wave_sync();
            w.template rows<true, true>(lds, lds + kBytes, table, table + 32, row0, at.len);
            gdr::wave_sync();
            reads_done();
        }
    w.finish(p, at, hk);
    if (w.key < at.len) w.store(p, at, hk);
}

// kWaves: on a SIMD, that the registers are divided for.
template <typename T, int D, int kWaves>
__global__ void __launch_bounds__(256, kWaves) attn_dkdv_kernel(BwdArgs<T> p)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(kRows);
    __shared__ __attribute__((aligned(16))) char lds[2][2][kBytes];     // [buffer][q, dy]
    __shared__ __attribute__((aligned(16))) float table[2][2][kRows];   // [buffer][lse, D]
    __shared__ int finite[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, hk;
    unit_of(p.seqs, p.B, p.Hk, p.chunk_k, false, blockIdx.x, slot, hk);
    const Place at = locate<kTile>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int first = at.at / kRows, last = (at.len + kRows - 1) / kRows;
    const int h0 = hk * p.group, h_end = h0 + p.group;
    Copy<T, D, kRows, 4> cq, cy;
    cq.init(p.q_stride, wave, lane);
    cy.init(p.Hq * D, wave, lane);
    const unsigned base = lds_address(lds);
    f32x2 ahead;
    auto issue = [&](int buffer, int h, int block) __attribute__((always_inline)) {
        const int row0 = block * kRows, rows = at.len - row0;
        cq.issue(base + buffer * 2 * kBytes, p.q + (at.tok + row0) * p.q_stride + h * D, rows, wave, lane);
        cy.issue(base + buffer * 2 * kBytes + kBytes, p.dy + ((at.tok + row0) * p.Hq + h) * D, rows, wave, lane);
        if (wave == 0) {   // rows that are not there have no weights
            ahead = f32x2{-kNegInf, 0.f};
            if (lane < rows) ahead = p.stats[h * p.tokens + at.tok + row0 + lane];
        }
    };
    // From the last rows to the first, and head by head within: so the workgroups
    // of a key head, which start together, read the same rows at the same time.
    // Waits for the next block of rows and sends for the one behind it.
    int buffer = 1, block = last - 1, h = h0, row0 = 0;
    auto arrive = [&]() __attribute__((always_inline)) {
        buffer ^= 1;
        row0 = block * kRows;
        wait_dma();
        if (wave == 0) {
            table[buffer][0][lane] = ahead[0];
            table[buffer][1][lane] = ahead[1];
        }
        __syncthreads();
        if (++h == h_end) {
            h = h0;
            --block;
        }
        if (block >= first) issue(buffer ^ 1, h, block);
    };
    issue(0, h0, block);
    const int key0 = at.at + 32 * wave;
    Keys<T, D> w;
    w.init(p, at, hk, key0, lane);
    while (block >= first + kTile / kRows) {   // these rows see every key
        arrive();
#pragma unroll
        for (int t = 0; t < 2; ++t)
            w.template rows<false, false>(lds[buffer][0] + L::bytes(32) * t, lds[buffer][1] + L::bytes(32) * t,
                                          &table[buffer][0][32 * t], &table[buffer][1][32 * t], row0 + 32 * t, at.len);
    }
    while (block >= first) {
        arrive();
        for (int t = 0; t < 2; ++t)
            if (row0 + 32 * t + 31 >= key0 && key0 < at.len)
                w.template rows<true, false>(lds[buffer][0] + L::bytes(32) * t, lds[buffer][1] + L::bytes(32) * t,
                                             &table[buffer][0][32 * t], &table[buffer][1][32 * t], row0 + 32 * t,
                                             at.len);
    }
    if (!all_waves(all_finite(w.dk) && all_finite(w.dv), finite, wave, lane)) {
        if (key0 < at.len) careful_keys<T, D>(p, at, hk, key0, lds[wave >> 1][wave & 1], table[wave >> 1][wave & 1]);
        return;
    }
    if (w.key < at.len) w.store(p, at, hk);
}

// The sum of the four waves' results, by rows of `count` tokens, times `by`.
template <typename T, int D, int kWave>
__device__ __forceinline__ void join(const char (&lds)[4][kWave], T *out, int64_t stride, int count, float by)
{
    constexpr int kLanes = D / 4;
    const int col = 4 * (threadIdx.x % kLanes);
    for (int i = threadIdx.x / kLanes; i < count; i += 256 / kLanes) {
        const f32x4 x = (get_row<D>(lds[0], i, col) + get_row<D>(lds[1], i, col)) +
                        (get_row<D>(lds[2], i, col) + get_row<D>(lds[3], i, col));
        *reinterpret_cast<Quad<T> *>(out + i * stride + col) = __builtin_convertvector(x * by, Quad<T>);
    }
}

// The narrow form: a wave has every fourth 32 rows of all the heads.
// With heads of 64 in bf16 the registers are divided for two waves on a SIMD: divided
// for one, matrix results go by way of the other half of the registers.  The whole
// backward, us, for one and two: 1 x 8192, 8 / 1 heads 802 and 730; 1 x 2048, 8 / 8 51 and
// 46; 4 x 2000, 12 / 3 192 and 133; 3000 tokens in 9 sequences, 16 / 4 57 and 53.
template <typename T, int D>
__global__ void __launch_bounds__(256, (sizeof(T) == 2 && D == 64 ? 2 : 1)) attn_dkdv_narrow_kernel(BwdArgs<T> p)
{
    using O = Own<T, D>;
    __shared__ __attribute__((aligned(16))) char lds[4][O::kWave];
    __shared__ __attribute__((aligned(16))) float table[4][2][32];   // lse, D
    __shared__ int finite[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, hk;
    unit_of(p.seqs, p.B, p.Hk, p.chunk_k, false, blockIdx.x, slot, hk);
    const Place at = locate<kNarrow>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int first = at.at / 32, per = (at.len + 31) / 32 - first;
    const int steps = per * p.group;   // fits: few workgroups of kTile keys, so few tokens
    Copy<T, D, 32, 1> cq, cy;
    cq.init(p.q_stride, 0, lane);
    cy.init(p.Hq * D, 0, lane);
    const unsigned base = lds_address(lds[wave]);
    f32x2 ahead;
    auto send = [&](int n) __attribute__((always_inline)) {
        const int g = n / per, h = hk * p.group + g, row0 = (first + n - g * per) * 32, rows = at.len - row0;
        const unsigned to = base + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
        cq.issue(to, p.q + (at.tok + row0) * p.q_stride + h * D, rows, 0, lane);
        cy.issue(to + O::kBytes, p.dy + ((at.tok + row0) * p.Hq + h) * D, rows, 0, lane);
        ahead = f32x2{-kNegInf, 0.f};   // rows that are not there have no weights
        if ((lane & 31) < rows) ahead = p.stats[h * p.tokens + at.tok + row0 + (lane & 31)];
    };
    if (wave < steps) send(wave);
    Keys<T, D> w;
    w.init(p, at, hk, at.at, lane);
    for (int n = wave; n < steps; n += 4) {
        wait_dma();
        table[wave][lane >> 5][lane & 31] = ahead[lane >> 5];
        gdr::wave_sync();
        if (O::kBuffers == 2 && n + 4 < steps) send(n + 4);
        const char *qy = lds[wave] + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
        const int at_row = n % per;
        if (at_row == 0)
            w.template rows<true, false>(qy, qy + O::kBytes, table[wave][0], table[wave][1], first * 32, at.len);
        else
            w.template rows<false, false>(qy, qy + O::kBytes, table[wave][0], table[wave][1], (first + at_row) * 32, at.len);
        gdr::wave_sync();
        reads_done();
        if (O::kBuffers == 1 && n + 4 < steps) send(n + 4);
    }
    if (!all_waves(all_finite(w.dk) && all_finite(w.dv), finite, wave, lane)) {
        if (wave == 0) careful_keys<T, D>(p, at, hk, at.at, lds[0], table[0][0]);
        return;
    }
    const int count = at.len - at.at < kNarrow ? at.len - at.at : kNarrow;
    const int64_t to = ((at.tok + at.at) * p.Hk + hk) * D;
    put_rows<D>(lds[wave], w.dk, lane);
    __syncthreads();
    join<T, D>(lds, p.dk + to, p.Hk * D, count, p.scale);
    __syncthreads();
    put_rows<D>(lds[wave], w.dv, lane);
    __syncthreads();
    join<T, D>(lds, p.dv + to, p.Hk * D, count, 1.f);
}

// 32 rows of a wave.
template <typename T, int D>
struct Rows {
    Tile<T, D> tl;
    Oct<T> q[D / 16], dy[D / 16];
    f32x16 dq[D / 32];
    f32x2 st;
    float c;
    int row0, row, half;

    // `leave`: into the table too.
    __device__ __forceinline__ void init(const BwdArgs<T> &p, const Place &at, int h, int first, int lane, bool leave)
    {
        tl.init(lane);
        half = lane >> 5;
        row0 = first;
        row = row0 + (lane & 31);
        const int64_t r = at.tok + (row < at.len ? row : at.len - 1);
        const T *qp = p.q + r * p.q_stride + h * D + 8 * half, *yp = p.dy + (r * p.Hq + h) * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            q[ks] = *reinterpret_cast<const Oct<T> *>(qp + 16 * ks);
            dy[ks] = *reinterpret_cast<const Oct<T> *>(yp + 16 * ks);
        }
        const int64_t e = (r * p.Hq + h) * D + 8 * half;
        float d = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const f32x8 a = wide<T>(dy[ks]);
            f32x8 y = wide<T>(*reinterpret_cast<const Oct<T> *>(p.y + e + 16 * ks));
            if (sizeof(T) == 2 && p.record) y += wide<bf16>(*reinterpret_cast<const bf16x8 *>(p.record + e + 16 * ks));
#pragma unroll
            for (int j = 0; j < 8; ++j) d = fmaf(a[j], y[j], d);
        }
        st = f32x2{p.lse[r * p.Hq + h] * kLog2e, half_sum(d)};
        if (leave && half == 0 && row < at.len) p.stats[h * p.tokens + r] = st;
        c = p.scale * kLog2e;
        clear();
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) dq[dt] = zero16();
    }
    // 32 keys from key0 on; kMask where some row may not see all of them: the tile that
    // begins with the wave's first row is cut through.
    template <bool kMask, bool kCareful>
    __device__ __forceinline__ void keys(const char *kt, const char *vt, int key0)
    {
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
            for (int dt = 0; dt < D / 32; ++dt) {
                Oct<T> x = tl.col(kt, dt, ss);
                if (kCareful && kMask && key0 == row0) x = finite_of<T>(x);
                dq[dt] = mma(x, w, dq[dt]);
            }
        }
    }
    // After the last of them, with care: what was left out of the tile that is cut through.
    // (A k that is not finite makes the score, and so the row's sum or its own weight.)
    __device__ __forceinline__ void finish(const T *kp, int64_t stride, int len)
    {
        int own = row;
        asm volatile("" : "+v"(own));   // else a register holds row - row0 from the start
        add_odd<T, D, true>(dq, kp + row0 * stride, stride, len - row0 < 32 ? len - row0 : 32, (2u << (own - row0)) - 1,
                            half);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) attn_dq_kernel(BwdArgs<T> p)
{
    using L = Tile<T, D>;
    constexpr int kBytes = L::bytes(kRows);
    __shared__ __attribute__((aligned(16))) char lds[2][2][kBytes];   // [buffer][k, v]
    __shared__ int finite[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, h;
    unit_of(p.seqs, p.B, p.Hq, p.chunk_q, true, blockIdx.x, slot, h);
    const Place at = locate<kTile>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int hk = h / p.group;
    const T *kp = uniform(p.k + at.tok * p.k_stride + hk * D), *vp = uniform(p.v + at.tok * p.v_stride + hk * D);
    const int end = at.at + kTile < at.len ? at.at + kTile : at.len;
    const int blocks = (end + kRows - 1) / kRows;
    Copy<T, D, kRows, 4> ck, cv;
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
    r.init(p, at, h, row0, lane, true);
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
    auto pass = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(careful)::value;
        int n = 0;
        for (; n < at.at / kRows; ++n) {   // every row sees all of these
            const auto *kv = arrive(n);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                r.template keys<false, kCareful>(kv[0] + L::bytes(32) * t, kv[1] + L::bytes(32) * t, n * kRows + 32 * t);
        }
        for (; n < blocks; ++n) {
            const auto *kv = arrive(n);
            for (int t = 0; t < 2; ++t)
                if (n * kRows + 32 * t <= row0 + 31 && row0 < at.len)
                    r.template keys<true, kCareful>(kv[0] + L::bytes(32) * t, kv[1] + L::bytes(32) * t,
                                                    n * kRows + 32 * t);
        }
    };
    pass(std::false_type{});
    if (!all_waves(all_finite(r.dq), finite, wave, lane)) {
        first();
        r.clear();
        pass(std::true_type{});
        if (row0 < at.len) r.finish(kp, p.k_stride, at.len);
    }
    if (r.row >= at.len) return;
    const int64_t to = ((at.tok + r.row) * p.Hq + h) * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 x = f32x4{r.dq[dt][i], r.dq[dt][i + 1], r.dq[dt][i + 2], r.dq[dt][i + 3]} * p.scale;
            *reinterpret_cast<Quad<T> *>(p.dq + to + 32 * dt + reg_row(i, r.half)) = __builtin_convertvector(x, Quad<T>);
        }
}

// The narrow form: a wave has every fourth 32 keys.
template <typename T, int D>
__global__ void __launch_bounds__(256, 1) attn_dq_narrow_kernel(BwdArgs<T> p)
{
    using O = Own<T, D>;
    __shared__ __attribute__((aligned(16))) char lds[4][O::kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int slot, h;
    unit_of(p.seqs, p.B, p.Hq, p.chunk_q, true, blockIdx.x, slot, h);
    const Place at = locate<kNarrow>(p.seqs, slot, lane);
    if (at.len == 0) return;
    const int hk = h / p.group;
    const T *kp = uniform(p.k + at.tok * p.k_stride + hk * D), *vp = uniform(p.v + at.tok * p.v_stride + hk * D);
    Copy<T, D, 32, 1> ck, cv;
    ck.init(p.k_stride, 0, lane);
    cv.init(p.v_stride, 0, lane);
    const unsigned base = lds_address(lds[wave]);
    const int last = at.at / 32;
    auto send = [&](int n) __attribute__((always_inline)) {
        const unsigned to = base + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
        const int64_t first = (int64_t)n * 32;
        ck.issue(to, kp + first * p.k_stride, at.len - (int)first, 0, lane);
        cv.issue(to + O::kBytes, vp + first * p.v_stride, at.len - (int)first, 0, lane);
    };
    if (wave <= last) send(wave);
    Rows<T, D> r;
    r.init(p, at, h, at.at, lane, wave == 0);
    auto pass = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool kCareful = decltype(careful)::value;
        for (int n = wave; n <= last; n += 4) {
            wait_dma();
            if (O::kBuffers == 2 && n + 4 <= last) send(n + 4);
            const char *kv = lds[wave] + (O::kBuffers == 2 ? (n >> 2 & 1) * 2 * O::kBytes : 0);
            if (n < last)
                r.template keys<false, kCareful>(kv, kv + O::kBytes, n * 32);
            else
                r.template keys<true, kCareful>(kv, kv + O::kBytes, n * 32);
            reads_done();
            if (O::kBuffers == 1 && n + 4 <= last) send(n + 4);
        }
    };
    pass(std::false_type{});
    if (!all_finite(r.dq)) {   // (a wave by itself)
        send(wave);
        r.clear();
        pass(std::true_type{});
        if (last % 4 == wave) r.finish(kp, p.k_stride, at.len);
    }
    put_rows<D>(lds[wave], r.dq, lane);
    __syncthreads();
    const int count = at.len - at.at < kNarrow ? at.len - at.at : kNarrow;
    join<T, D>(lds, p.dq + ((at.tok + at.at) * p.Hq + h) * D, p.Hq * D, count, p.scale);
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
    const int64_t bytes = a.seqs.T * 2 * D * (int64_t)sizeof(T);   // of k and v, or q and dy, of a head
    p.chunk_q = chunk_of(a.seqs, a.seqs.starts ? a.Hq : a.B * a.Hq, bytes, p.group);
    p.chunk_k = chunk_of(a.seqs, a.seqs.starts ? a.Hk : a.B * a.Hk, bytes * p.group, 1);
    BwdArgs<T> few = p;
    few.seqs = narrow(a.seqs, a.B);
    if (is_narrow(a.seqs.slots * a.Hq, a.dtype))
        hipLaunchKernelGGL((attn_dq_narrow_kernel<T, D>), dim3((unsigned)(few.seqs.slots * a.Hq)), dim3(256), 0, stream,
                           few);
    else
        hipLaunchKernelGGL((attn_dq_kernel<T, D>), dim3((unsigned)(a.seqs.slots * a.Hq)), dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // With heads of 64 in bf16, room for a third workgroup on a compute unit pays where
    // there are enough of them: the whole backward, us, two and three, 1 x 4096 x 24 heads
    // (768) 206 and 215, 1 x 4096 x 32 (1024) 268 and 259, 4 x 4096 x 32 (4096) 1018 and 963.
    constexpr bool kThree = sizeof(T) == 2 && D == 64;
    const int64_t keys = a.seqs.slots * a.Hk;
    if (is_narrow(keys, a.dtype))
        hipLaunchKernelGGL((attn_dkdv_narrow_kernel<T, D>), dim3((unsigned)(few.seqs.slots * a.Hk)), dim3(256), 0, stream,
                           few);
    else if (kThree && keys >= 1024)
        hipLaunchKernelGGL((attn_dkdv_kernel<T, D, kThree ? 3 : 1>), dim3((unsigned)keys), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((attn_dkdv_kernel<T, D, kThree ? 2 : 1>), dim3((unsigned)keys), dim3(256), 0, stream, p);
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
