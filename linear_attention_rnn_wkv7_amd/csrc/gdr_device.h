// Device-side pieces of the gated delta rule's chunk kernels (gfx950).
//
// The chunk form.  Over a chunk of C = 64 tokens with inclusive log-decay sums
// G_i, gamma_i = exp(G_i), Gamma_ij = exp(G_i - G_j), and the state S0 (here
// [K][V]) before it:
//     R = V - gamma * (K S0)                         [C, V]
//     E = T R,  T = (I + N diag(beta))^-1,  N_ij = Gamma_ij k_i . k_j  (i > j)
//     Y = gamma * (Q S0) + P E,  P_ij = beta_j Gamma_ij q_i . k_j      (i >= j)
//     S1 = gamma_C S0 + K^T W,  W_j = (gamma_C / gamma_j) beta_j E_j
// (E_j is what token j's value differs from what the state answers to k_j.)
// No exponent is ever positive while g <= 0, and no division occurs.
//
// Operands.  Everything runs on 16 x 16 matrix tiles.  A tile's result has
// its rows on (lane / 16, register) and its columns on lane % 16; as an
// operand of the next product, contracted over those rows, it needs no lane
// exchange if the other operand supplies its k values in the same order:
// position 8 (lane / 16) + j of a 32-deep step stands for
//     k = 16 (j / 4) + 4 (lane / 16) + j % 4.
// Arrays in LDS that serve as the other operand are stored in that order, so
// a lane's 8 values are contiguous.  A 16-column slab of the state thus runs
// through K S0, T R, P E and K^T W inside one wave, with no barrier.
//
// fp32 inputs use the fp32 matrix instruction (8 per 32-deep step).  With
// bf16 inputs, q, k, v, dy are exact operands, and every fp32 operand is
// carried as kParts bf16 parts x = x0 + x1 + .. (each the rounding of what
// is left), of whose products those above 2^-8 kParts are formed.  That holds
// for what y alone is made of too: y is the difference of large terms where a
// token reads a key that has been written again, and two parts, 2^-16 of each
// term, would then be worse than y's own rounding (a state 4096 times as large
// as the value in its place: 15 half steps of bf16 and more).
#pragma once

#include "gdr_internal.h"
#include "wkv7_device.h"

namespace wkv7 {
namespace gdr {

using bf16 = __bf16;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Num;
template <>
struct Num<float> {
    static constexpr int kPlanes = 1;
    using Quad = f32x4;
    using Oct = f32x8;
};
template <>
struct Num<bf16> {
    static constexpr int kPlanes = kParts;
    using Quad = bf16x4;
    using Oct = bf16x8;
};

// The stored position of k inside its 32-deep step.
__device__ __forceinline__ int kpos(int k)
{
    return (k & ~31) | ((k >> 2) & 3) << 3 | ((k >> 4) & 1) << 2 | (k & 3);
}

// Eight k values of one row (or column) per lane, in P parts.
template <typename T, int P>
struct Frag {
    typename Num<T>::Oct p[P];
};

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Products of parts i + j >= kParts are left out.
template <int PA, int PB>
__device__ __forceinline__ f32x4 mma(f32x4 c, const Frag<bf16, PA> &a, const Frag<bf16, PB> &b)
{
#pragma unroll
    for (int i = PA - 1; i >= 0; --i)
#pragma unroll
        for (int j = PB - 1; j >= 0; --j)
            if (i + j < kParts) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], c, 0, 0, 0);
    return c;
}
template <int PA, int PB>
__device__ __forceinline__ f32x4 mma(f32x4 c, const Frag<float, PA> &a, const Frag<float, PB> &b)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.p[0][j], b.p[0][j], c, 0, 0, 0);
    return c;
}

// Two floats rounded to bf16, the first in the low half: one conversion (the
// empty asm keeps the compiler from converting each value by itself and
// packing afterwards).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    asm("" : "+v"(u));
    return u;
}

// kN floats as P parts: x[p] takes part p, pairs packed.
template <int kN, int P>
__device__ __forceinline__ void split(float (&v)[kN], uint32_t (&x)[P][kN / 2])
{
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            x[p][i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            if (p + 1 < P) {
                v[2 * i] -= bf16_lo(x[p][i]);
                v[2 * i + 1] -= bf16_hi(x[p][i]);
            }
        }
}

// Four values as P parts of an operand's quad.
template <typename T, int P>
__device__ __forceinline__ void split_quad(f32x4 x, typename Num<T>::Quad (&q)[P])
{
    if constexpr (sizeof(T) == 4) {
        q[0] = x;
    } else {
        float v[4] = {x[0], x[1], x[2], x[3]};
        uint32_t u[P][2];
        split(v, u);
#pragma unroll
        for (int p = 0; p < P; ++p) __builtin_memcpy(&q[p], u[p], 8);
    }
}

// Two result tiles (rows 0..15 and 16..31 of a step) as one operand.
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> make_frag(f32x4 lo, f32x4 hi)
{
    Frag<T, P> f;
    if constexpr (sizeof(T) == 4) {
        f.p[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        uint32_t u[P][4];
        split(v, u);
#pragma unroll
        for (int p = 0; p < P; ++p) __builtin_memcpy(&f.p[p], u[p], 16);
    }
    return f;
}

// The lane number, or an offset made from it, fresh to the compiler: in a loop
// it otherwise keeps everything computed from it in registers of its own.
__device__ __forceinline__ uint32_t fresh(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// Chunk operands that are copied straight into LDS, [64][K] by rows, cannot
// be padded; the 16-byte pieces of row t are permuted instead, piece p at
// p ^ swizzle(t), so that neither 16 rows' reads of one piece nor 8 rows' of
// two meet a bank twice.
template <typename T, int K>
struct Swizzled {
    static constexpr int kRowBytes = K * (int)sizeof(T), kPieces = kRowBytes / 16, kBytes = 64 * kRowBytes;

    __device__ static __forceinline__ int swizzle(int t)
    {
        return kPieces == 8 ? ((t >> 1) & 3) << 1 | ((t >> 3) & 1) : (t & 7) << 1 | ((t >> 3) & 1);
    }
    __device__ static __forceinline__ int at(int t, int byte)
    {
        return t * kRowBytes + (((byte >> 4) ^ swizzle(t)) << 4 | (byte & 15));
    }
    // Row 16 it + l16 as an operand: k = 32 ks + the order above.
    __device__ static __forceinline__ Frag<T, 1> rows(const char *lds, int it, int ks, int lg, int l16)
    {
        using Quad = typename Num<T>::Quad;
        const int b = (32 * ks + 4 * lg) * (int)sizeof(T);
        const char *r = lds + 16 * it * kRowBytes;
        const Quad lo = *reinterpret_cast<const Quad *>(r + at(l16, b));
        const Quad hi = *reinterpret_cast<const Quad *>(r + at(l16, b + 16 * (int)sizeof(T)));
        Frag<T, 1> f;
        f.p[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return f;
    }
    // Column 16 i + l16 as an operand, k = tokens 32 ks + the order above.
    // bf16: the transposing LDS read hands each 16 lanes' 4 x 16 block (row
    // l16 / 4, four columns to a lane) out by columns.
    __device__ static __forceinline__ Frag<T, 1> cols(const char *lds, int i, int ks, int lg, int l16)
    {
        Frag<T, 1> f;
        if constexpr (sizeof(T) == 2) {
            typename Num<T>::Quad x[2];
            const int t = 4 * lg + (l16 >> 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char *p = lds + (32 * ks + 16 * h) * kRowBytes + at(t, 32 * i + 8 * (l16 & 3));
                x[h] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                    (__attribute__((address_space(3))) bf16x4 *)(const __attribute__((address_space(3))) char *)p);
            }
            f.p[0] = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.p[0][j] = *reinterpret_cast<const float *>(lds + (32 * ks + 16 * (j >> 2)) * kRowBytes +
                                                             at(4 * lg + (j & 3), 64 * i + 4 * l16));
        }
        return f;
    }
};

// Copies by one wave straight into LDS (1 KB per instruction); complete after
// wait_dma() and a barrier.  A swizzled operand, rows `stride` elements apart
// (a multiple of K); rows behind the last of `len` repeat it (their weights
// are zero).
template <typename T, int K>
__device__ __forceinline__ void dma_rows(char *lds, const T *src, int64_t stride, int len, int lane)
{
    using S = Swizzled<T, K>;
    constexpr int kRows = 64 / S::kPieces;   // rows per copy
    const unsigned to = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const int row = lane / S::kPieces, piece = lane % S::kPieces;
    const uint32_t step = (uint32_t)(stride * (int64_t)sizeof(T));
    if (len == kChunk) {
        // swizzle() only moves bits: that of n * kRows + row is the exclusive or
        const uint32_t off = row * step + ((piece ^ S::swizzle(row)) << 4);
        const char *base = reinterpret_cast<const char *>(src);
#pragma unroll
        for (int n = 0; n < S::kBytes / 1024; ++n, base += kRows * step)
            dma16_split(base, off ^ (S::swizzle(n * kRows) << 4), to + n * 1024);
    } else {
        for (int n = 0; n < S::kBytes / 1024; ++n) {
            const int t = n * kRows + row, u = t < len ? t : len - 1;
            dma16_split(src, u * step + ((piece ^ S::swizzle(t)) << 4), to + n * 1024);
        }
    }
}
template <int kBytes>
__device__ __forceinline__ void dma_flat(void *lds, const void *src, int lane)
{
    static_assert(kBytes % 1024 == 0, "whole copies");
    const unsigned to = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
#pragma unroll
    for (int n = 0; n < kBytes / 1024; ++n)
        dma16_split(static_cast<const char *>(src) + n * 1024, lane * 16, to + n * 1024);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return (float)x; }
__device__ __forceinline__ f32x4 quad_f32(f32x4 x) { return x; }
__device__ __forceinline__ f32x4 quad_f32(bf16x4 x) { return __builtin_convertvector(x, f32x4); }

// A chunk slot's first token (in the [B * T] token list) and its length.
struct Chunk {
    int64_t tok;
    int len;
};

__device__ __forceinline__ void seq_range(const Map &m, int64_t s, int64_t &lo, int64_t &hi)
{
    if (!m.starts) {   // a row, or a segment of one
        const int64_t row = s / m.nseg, at = s % m.nseg * m.nckseg * kChunk;
        lo = row * m.T + at;
        hi = at + m.nckseg * kChunk < m.T ? lo + m.nckseg * kChunk : (row + 1) * m.T;
        return;
    }
    lo = m.starts[s];
    hi = m.starts[s + 1];
    lo = lo < 0 ? 0 : lo > m.T ? m.T : lo;
    hi = hi < lo ? lo : hi > m.T ? m.T : hi;
}

// The slot of a sequence's first chunk.  Packed sequence s starts at slot
// floor(start / 64) + s: ceil(len / 64) <= floor(end / 64) - floor(start / 64)
// + 1 keeps the sequences' slots apart and below T / 64 + nseq without a sum
// over the sequences before.
__device__ __forceinline__ int64_t first_slot(const Map &m, int64_t s, int64_t lo)
{
    return m.starts ? lo / kChunk + s : s / m.nseg * m.nck + s % m.nseg * m.nckseg;
}

__device__ __forceinline__ Chunk locate(const Map &m, int64_t slot)
{
    Chunk c;
    int64_t lo, hi, at;
    if (!m.starts) {
        const int64_t row = slot / m.nck;
        lo = row * m.T;
        hi = lo + m.T;
        at = slot - row * m.nck;
    } else {
        int64_t a = 0, b = m.nseq - 1;   // the last sequence whose first slot is <= slot
        while (a < b) {
            const int64_t mid = (a + b + 1) >> 1;
            seq_range(m, mid, lo, hi);
            if (first_slot(m, mid, lo) <= slot)
                a = mid;
            else
                b = mid - 1;
        }
        seq_range(m, a, lo, hi);
        at = slot - first_slot(m, a, lo);
    }
    c.tok = lo + at * kChunk;
    const int64_t left = hi - c.tok;
    c.len = at < 0 || left <= 0 ? 0 : left < kChunk ? (int)left : kChunk;
    return c;
}

// Four rows i0 .. of one kind of a chunk's table.
__device__ __forceinline__ f32x4 row4(const float *tab, int kind, int i0)
{
    return *reinterpret_cast<const f32x4 *>(tab + kind * 64 + i0);
}

// Between a wave's own LDS writes and its other lanes' reads of them.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Sum over the 64 lanes, in every lane.
template <typename F>
__device__ __forceinline__ F wave_sum(F x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

}  // namespace gdr
}  // namespace wkv7
