// Device-side pieces of the attention kernels (gfx950).
//
// Everything runs on 32 x 32 matrix tiles.  A result tile has its column on
// lane % 32 and, of its rows, 8 (i / 4) + 4 (lane / 32) + i % 4 in register i.
// Operands give a lane 8 values of one row (or column), lane % 32, for each
// 16-deep step.  The products of queries and keys are formed as K Q^T (or Q K^T
// for the gradients of k and v), so that the softmax's row, or the key, is a
// lane: its maximum and sum stay in the lane and its other half (lane ^ 32).
// The weights are then, as they lie, the right operand of the next product,
// contracted over the tile's rows, if the left operand supplies its 16 values
// of a step in the same order:
//     position 8 (lane / 32) + j stands for 8 (j / 4) + 4 (lane / 32) + j % 4.
// The transposing LDS read gives that order, so no weight ever leaves its lane.
// fp32 inputs run the same code on the fp32 matrix instruction (8 per step).
#pragma once

#include "attn_internal.h"
#include "gdr_device.h"

namespace wkv7 {
namespace attn {

using gdr::bf16;
using gdr::bf16x2;
using gdr::bf16x4;
using gdr::bf16x8;
using gdr::f32x2;
using gdr::f32x4;
using gdr::f32x8;
using gdr::pack_bf16;
using gdr::to_f32;
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_huge_valf();
// Where a running maximum starts: below every score, and 0 away from itself, so
// that scores of minus infinity have weight 0 before there is another.
constexpr float kLowest = -__FLT_MAX__;

template <typename T>
using Oct = typename gdr::Num<T>::Oct;
template <typename T>
using Quad = typename gdr::Num<T>::Quad;

__device__ __forceinline__ f32x16 zero16()
{
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    return x;
}
template <typename T>
__device__ __forceinline__ Oct<T> zero_oct()
{
    Oct<T> x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)0.f;
    return x;
}

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x8 a, f32x8 b, f32x16 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// Result registers 8 s .. 8 s + 7 as the operand of step s.
template <typename T>
__device__ __forceinline__ Oct<T> as_operand(const f32x16 &x, int s)
{
    Oct<T> o;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = x[8 * s + j];
    } else {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = pack_bf16(x[8 * s + 2 * j], x[8 * s + 2 * j + 1]);
        __builtin_memcpy(&o, u, 16);
    }
    return o;
}

// The row of a result register.
__device__ __forceinline__ int reg_row(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

// x of the lane and of its other half (lane ^ 32).  (The empty asm: see swap_add32.)
struct Halves {
    float a, b;
};
__device__ __forceinline__ Halves both_halves(float x)
{
    auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x),
                                              false, false);
    unsigned lo = p[0], hi = p[1];
    asm volatile("" : "+v"(hi));
    return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float half_max(float x)
{
    const Halves h = both_halves(x);
    return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float half_sum(float x)
{
    const Halves h = both_halves(x);
    return h.a + h.b;
}

// A pointer that is the same in all lanes, into scalar registers (what is made of it in
// loops is else vector arithmetic as soon as it lives past them).
template <typename T>
__device__ __forceinline__ const T *uniform(const T *p)
{
    typedef const __attribute__((address_space(1))) T *Global;
    const uint64_t b = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b), hi = __builtin_amdgcn_readfirstlane((int)(b >> 32));
    return (const T *)(Global)((uintptr_t)((uint64_t)hi << 32 | lo));
}

// Rows of D entries in LDS, in 16-byte pieces, 64 of them to a group: what one
// copy straight into LDS lays end to end.  Groups are 16 or 32 bytes apart, and
// piece p of row t lies at p ^ x(t) in its row: so the 16 rows that a read of one
// piece of 32 rows takes at a time (those with (t / 4) % 8 among 0, 3, 5, 6, then
// the others) meet each bank once, and so do the transposing read's 4 rows of four
// pieces, while a lane's address is one of a few, made once, and a constant.
template <typename T, int D>
struct Tile {
    static constexpr int kPitch = D * (int)sizeof(T), kPieces = kPitch / 16, kPerCopy = 64 / kPieces;
    static constexpr int kGroup = 1024 + (kPieces == 8 ? 32 : 16);
    static constexpr int bytes(int rows) { return rows / kPerCopy * kGroup; }

    __device__ static __forceinline__ int x(int t)
    {
        if (kPieces == 8) return ((t >> 1) & 1) << 2 | ((t >> 2) & 1);
        if (kPieces == 16) return (t & 3) << 2;
        return (t & 1) << 3;
    }
    __device__ static __forceinline__ int at(int t, int piece)
    {
        return t / kPerCopy * kGroup + t % kPerCopy * kPitch + ((piece ^ x(t)) << 4);
    }

    static constexpr int kRowBases = kPieces == 32 ? 2 : 4;
    static constexpr int kColBases = sizeof(T) == 2 ? D / 32 : kPieces == 32 ? 2 : 4;
    int row_base[kRowBases], col_base[kColBases];
    __device__ __forceinline__ void init(int lane)
    {
        const int l32 = lane & 31, half = lane >> 5;
        const int step = sizeof(T) == 2 && kPieces == 8 ? 2 : kPieces == 32 ? 8 : 4;   // pieces from a base to the next
#pragma unroll
        for (int i = 0; i < kRowBases; ++i) row_base[i] = at(l32, step * i + half * (int)sizeof(T) / 2);
#pragma unroll
        for (int i = 0; i < kColBases; ++i) {
            if (sizeof(T) == 2) {
                const int c = 2 * (lane & 16) + 8 * (lane & 3);
                col_base[i] = at(4 * half + ((lane >> 2) & 3), 4 * i + (c >> 4)) + (c & 15);
            } else {
                col_base[i] = at(4 * half, (l32 >> 2) ^ (kPieces == 32 ? 8 : 4) * i) + 4 * (lane & 3);
            }
        }
    }

    // Row lane % 32 of `lds` as an operand: entries 16 ks + 8 half ..
    __device__ __forceinline__ Oct<T> row(const char *lds, int ks) const
    {
        if constexpr (sizeof(T) == 2) {
            const int o = kPieces == 8 ? row_base[ks & 3] : row_base[(ks >> 1) & 3] + (ks & 1) * 32;
            return *reinterpret_cast<const bf16x8 *>(lds + o);
        } else {
            const int o = kPieces == 16 ? row_base[ks & 3]
                                        : row_base[(ks >> 1) & 1] + (ks & 1) * 64 + (ks >> 2) * 256;
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(lds + o);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(lds + o + 16);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Column 32 dt + lane % 32 as an operand: rows 16 s .. of `lds` in the order above.
    __device__ __forceinline__ Oct<T> col(const char *lds, int dt, int s) const
    {
        if constexpr (sizeof(T) == 2) {
            bf16x4 x[2];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const char *p = lds + col_base[dt] + (16 * s + 8 * jj) / kPerCopy * kGroup;
                x[jj] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (__attribute__((address_space(3))) bf16x4 *)(const __attribute__((address_space(3))) char *)p);
            }
            return __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            f32x8 x;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = 16 * s + 8 * (j >> 2) + (j & 3);
                const int o = t / kPerCopy * kGroup + t % kPerCopy * kPitch +
                              (kPieces == 16 ? col_base[(j & 3) ^ 2 * dt]
                                             : col_base[(j & 1) ^ (dt & 1)] + (dt >> 1) * 256);
                x[j] = *reinterpret_cast<const float *>(lds + o);
            }
            return x;
        }
    }
};

// Copies of N rows straight into LDS by the kWaves waves of a workgroup; they
// are complete after wait_dma() and a barrier.
template <typename T, int D, int N, int kWaves>
struct Copy {
    using L = Tile<T, D>;
    static constexpr int kEach = N / L::kPerCopy / kWaves;
    static_assert(kEach * kWaves * L::kPerCopy == N, "whole copies");
    uint32_t off;      // of this lane's piece from the first row of a copy
    uint32_t to;       // LDS address of the wave's first copy within the rows
    uint32_t stride;   // bytes

    __device__ __forceinline__ void init(int64_t stride_elements, int wave, int lane)
    {
        stride = (uint32_t)(stride_elements * (int64_t)sizeof(T));
        to = wave * kEach * L::kGroup;
        const int t = lane / L::kPieces;
        off = (uint32_t)t * stride + (((lane % L::kPieces) ^ L::x(t)) << 4);
    }
    // `rows` (at least one) of them are there; the others repeat the last.
    __device__ __forceinline__ void issue(unsigned lds, const T *src, int rows, int wave, int lane) const
    {
        const char *base = reinterpret_cast<const char *>(src);
        const int first = wave * kEach * L::kPerCopy;
        if (rows >= N) {
#pragma unroll
            for (int n = 0; n < kEach; ++n)
                dma16_split(base + (int64_t)(first + n * L::kPerCopy) * stride, off, lds + to + n * L::kGroup);
        } else {
#pragma unroll
            for (int n = 0; n < kEach; ++n) {
                const int t = first + n * L::kPerCopy + lane / L::kPieces, u = t < rows ? t : rows - 1;
                dma16_split(base, (uint32_t)u * stride + (((lane % L::kPieces) ^ L::x(t)) << 4),
                            lds + to + n * L::kGroup);
            }
        }
    }
    // Zeros for those that were not there, of what this wave has copied.
    __device__ __forceinline__ void clear(char *lds, int rows, int wave, int lane) const
    {
#pragma unroll
        for (int n = 0; n < kEach; ++n)
            if ((wave * kEach + n) * L::kPerCopy + lane / L::kPieces >= rows)
                *reinterpret_cast<f32x4 *>(lds + to + n * L::kGroup + lane * 16) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
};

__device__ __forceinline__ unsigned lds_address(const void *p)
{
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

__device__ __forceinline__ void seq_range(const Seqs &m, int64_t s, int64_t &lo, int64_t &hi)
{
    if (!m.starts) {
        lo = s * m.T;
        hi = lo + m.T;
        return;
    }
    lo = m.starts[s];
    hi = m.starts[s + 1];
    lo = lo < 0 ? 0 : lo > m.T ? m.T : lo;
    hi = hi < lo ? lo : hi > m.T ? m.T : hi;
}

// A tile: its sequence's first token (in the [B T] list) and length, and its
// own first token in the sequence.
struct Place {
    int64_t tok;
    int len, at;
};

// Tile `slot` of tiles of kRows tokens.  Packed sequence s starts at slot
// floor(start / kRows) + s: that keeps the sequences' slots apart and below T /
// kRows + nseq without a sum over the sequences before.  A slot behind its
// sequence's last tile has len = 0.  The last sequence whose first slot is not
// behind `slot` is found by the wave's lanes, 64 sequences (or ranges of them) at a time.
template <int kRows>
__device__ __forceinline__ Place locate(const Seqs &m, int slot, int lane)
{
    int64_t lo, hi;
    int at;
    if (!m.starts) {
        const int row = (uint32_t)slot / (uint32_t)m.tiles;
        lo = row * m.T;
        hi = lo + m.T;
        at = slot - row * (int)m.tiles;
    } else {
        const int nseq = (int)m.nseq;
        int first = 0, step = 1;
        while (step * 64 < nseq) step *= 64;
        for (; step; step /= 64) {
            const int s = first + lane * step;
            bool before = false;
            if (s < nseq) {
                const int start = m.starts[s];
                before = (start < 0 ? 0 : start > m.T ? (int)m.T : start) / kRows + s <= slot;
            }
            const int n = __popcll(__ballot(before));   // none: tokens before the first sequence
            first += (n > 0 ? n - 1 : 0) * step;
        }
        first = __builtin_amdgcn_readfirstlane(first);
        seq_range(m, first, lo, hi);
        at = slot - (int)(lo / kRows) - first;
    }
    const int64_t len = hi - lo;
    if (at < 0 || (int64_t)at * kRows >= len) return {lo, 0, 0};
    return {lo, (int)len, at * kRows};
}

// A wave's own tiles in a narrow workgroup: two arrays of 32 rows, twice where
// LDS has room.
template <typename T, int D>
struct Own {
    static constexpr int kBytes = Tile<T, D>::bytes(32);
    static constexpr int kBuffers = 4 * 2 * 2 * kBytes <= 140 * 1024 ? 2 : 1;
    // then the waves' results, by rows, are joined there
    static constexpr int kOut = 32 * (D + 4) * 4;
    static constexpr int kWave = kBuffers * 2 * kBytes > kOut ? kBuffers * 2 * kBytes : kOut;
};

// Between a wave's reads of LDS and copies to the same place.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A value that a row does not see has weight 0, which makes nothing of it if it is
// finite, and else NaN.  Only in the tile that the mask cuts through do some rows see
// what others do not.  So where a result has come out not finite, all is gone over once
// more with care: in that tile infinities and NaN stay out of the products, and the rows
// that see them get them at the end.  The loops that run else know nothing of this: what
// they pay is one look at the results, an instruction to two of them, and a barrier.
// Forward, us, without and with: 12288 tokens in 24 prompts, 32 / 8 heads of 128, 140 and
// 143; 16384 tokens, 32 / 4 heads of 64, 1120 and 1128.  Looking at the tile within the
// loop, or leaving such values out there: 148 to 150 for the prompts.

// Whether the wave's results are finite (the same in all lanes).
template <int N>
__device__ __forceinline__ bool all_finite(const f32x16 (&x)[N])
{
    float top = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(top, __builtin_fabsf(x[n][i]));
    return !__any(!(top < -kNegInf));
}
// Whether they are in all four waves, which have then all read what they read from LDS.
__device__ __forceinline__ bool all_waves(bool finite, int (&flags)[4], int wave, int lane)
{
    if (lane == 0) flags[wave] = finite;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(flags[0] & flags[1] & flags[2] & flags[3]);
}
// The lane's number for the pass with care: what is made of it is made anew where it is
// used, and takes no registers elsewhere.
__device__ __forceinline__ int lane_anew()
{
    uint32_t all = ~0u;
    asm volatile("" : "+s"(all));
    return (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}
// An operand with 0 for what is not finite.
template <typename T>
__device__ __forceinline__ Oct<T> finite_of(Oct<T> x)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __builtin_fabsf((float)x[j]) < -kNegInf ? x[j] : (T)0.f;
    return x;
}
// acc (by columns) += what is not finite of `rows` rows of `src`, as it is, or as NaN
// where its own score has made its weight NaN or 0; bit j of `sees`: whether the lane's
// column sees row j.
template <typename T, int D, bool kNan>
__device__ __forceinline__ void add_odd(f32x16 (&acc)[D / 32], const T *src, int64_t stride, int rows, uint32_t sees,
                                        int half)
{
#pragma unroll 1
    for (int j = 0; j < rows; ++j) {
        const bool seen = sees >> j & 1;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const Quad<T> x = *reinterpret_cast<const Quad<T> *>(src + j * stride + 32 * dt + reg_row(i, half));
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float y = (float)x[m];
                    if (seen && !(__builtin_fabsf(y) < -kNegInf)) acc[dt][i + m] += kNan ? __builtin_nanf("") : y;
                }
            }
    }
}

// A result by columns (its column on lane % 32) into LDS by rows of that, and the
// sum of the four waves' over them, in order.
template <int D>
__device__ __forceinline__ void put_rows(char *lds, const f32x16 (&x)[D / 32], int lane)
{
    float *out = reinterpret_cast<float *>(lds) + (lane & 31) * (D + 4);
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4 *>(out + 32 * dt + reg_row(i, lane >> 5)) =
                f32x4{x[dt][i], x[dt][i + 1], x[dt][i + 2], x[dt][i + 3]};
}
template <int D>
__device__ __forceinline__ f32x4 get_row(const char *lds, int row, int col)
{
    return *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(lds) + row * (D + 4) + col);
}

}  // namespace attn
}  // namespace wkv7
