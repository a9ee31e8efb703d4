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

// Rows of D entries in LDS, in 16-byte pieces.  Piece p of row t lies at p ^
// swizzle(t): 16 rows' reads of one piece meet each bank once, and so do the
// transposing read's 4 rows of four pieces.  (Rows cannot be padded: copies
// straight into LDS lay 64 pieces end to end.)
template <typename T, int D>
struct Tile {
    static constexpr int kPitch = D * (int)sizeof(T), kPieces = kPitch / 16, kPerCopy = 64 / kPieces;

    __device__ static __forceinline__ int swizzle(int t)
    {
        if (kPieces == 8) return ((t >> 1) & 1) << 2 | ((t >> 2) & 3);
        if (kPieces == 16) return (t & 3) << 2 | ((t >> 2) & 3);
        return t & 15;
    }
    __device__ static __forceinline__ int at(int t, int piece) { return t * kPitch + ((piece ^ swizzle(t)) << 4); }

    // Row lane % 32 of `lds` as an operand: entries 16 ks + 8 half ..
    __device__ static __forceinline__ Oct<T> row(const char *lds, int ks, int lane)
    {
        const int t = lane & 31, half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const bf16x8 *>(lds + at(t, 2 * ks + half));
        } else {
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(lds + at(t, 4 * ks + 2 * half));
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(lds + at(t, 4 * ks + 2 * half + 1));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Column 32 dt + lane % 32 as an operand: rows 16 s .. of `lds` in the order above.
    __device__ static __forceinline__ Oct<T> col(const char *lds, int dt, int s, int lane)
    {
        const int half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            bf16x4 x[2];
            const int t = 4 * half + ((lane >> 2) & 3), c = 2 * (lane & 31 & 16) + 8 * (lane & 3);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const char *p = lds + at(16 * s + 8 * jj + t, 4 * dt + (c >> 4)) + (c & 15);
                x[jj] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (__attribute__((address_space(3))) bf16x4 *)(const __attribute__((address_space(3))) char *)p);
            }
            return __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            f32x8 x;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = 16 * s + 8 * (j >> 2) + 4 * half + (j & 3);
                x[j] = *reinterpret_cast<const float *>(lds + at(t, 8 * dt + ((lane & 31) >> 2)) + 4 * (lane & 3));
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
    static constexpr int kCopies = N * L::kPitch / 1024, kEach = kCopies / kWaves;
    static_assert(kCopies % kWaves == 0, "whole copies");
    uint32_t off[kEach];   // of this lane's pieces from the first row
    uint32_t to;           // LDS address of the wave's first copy within the rows
    uint32_t stride;       // bytes

    __device__ __forceinline__ void init(int64_t stride_elements, int wave, int lane)
    {
        stride = (uint32_t)(stride_elements * (int64_t)sizeof(T));
        to = wave * kEach * 1024;
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const int t = (wave * kEach + n) * L::kPerCopy + lane / L::kPieces;
            off[n] = (uint32_t)t * stride + (((lane % L::kPieces) ^ L::swizzle(t)) << 4);
        }
    }
    // `rows` (at least one) of them are there; the others repeat the last.
    __device__ __forceinline__ void issue(unsigned lds, const T *src, int rows, int wave, int lane) const
    {
        if (rows >= N) {
#pragma unroll
            for (int n = 0; n < kEach; ++n) dma16_split(src, off[n], lds + to + n * 1024);
        } else {
#pragma unroll
            for (int n = 0; n < kEach; ++n) {
                const int t = (wave * kEach + n) * L::kPerCopy + lane / L::kPieces;
                const uint32_t back = t < rows ? 0 : (uint32_t)(t - rows + 1) * stride;
                dma16_split(src, off[n] - back, lds + to + n * 1024);
            }
        }
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

// Packed sequence s starts at slot floor(start / kTile) + s: that keeps the
// sequences' slots apart and below T / kTile + nseq without a sum over the
// sequences before.  A slot behind its sequence's last tile has at >= len.
__device__ __forceinline__ Place locate(const Seqs &m, int64_t slot)
{
    int64_t lo, hi, at;
    if (!m.starts) {
        const int64_t row = slot / m.tiles;
        lo = row * m.T;
        hi = lo + m.T;
        at = slot - row * m.tiles;
    } else {
        int64_t a = 0, b = m.nseq - 1;   // the last sequence whose first slot is <= slot
        while (a < b) {
            const int64_t mid = (a + b + 1) >> 1;
            seq_range(m, mid, lo, hi);
            if (lo / kTile + mid <= slot)
                a = mid;
            else
                b = mid - 1;
        }
        seq_range(m, a, lo, hi);
        at = slot - (lo / kTile + a);
    }
    const int64_t len = hi - lo;
    if (at < 0 || at * kTile >= len) return {lo, 0, 0};
    return {lo, (int)len, (int)(at * kTile)};
}

// Block -> (slot, head).  Rows' last tiles, which see the most, start first.
// Workgroups go to the 8 dies in turn: of the units (row, head) of one tile,
// neighbours, which read the same keys, go to one die, whose cache then holds
// them for all.
__device__ __forceinline__ void unit_of(const Seqs &m, int64_t B, int64_t heads, bool last_first, int64_t id,
                                        int64_t &slot, int64_t &head)
{
    const int64_t units = m.starts ? heads : B * heads;
    int64_t tile = id / units, u = id - tile * units;
    if (units % 8 == 0) u = u % 8 * (units / 8) + u / 8;
    const int64_t tiles = m.starts ? m.slots : m.tiles;
    if (last_first) tile = tiles - 1 - tile;
    head = u % heads;
    slot = m.starts ? tile : u / heads * m.tiles + tile;
}

}  // namespace attn
}  // namespace wkv7
