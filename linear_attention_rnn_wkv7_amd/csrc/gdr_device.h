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
// is left), of whose products those above 2^-8 kParts are formed.
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

// LDS row padding: 16 bytes, so that 16 rows' 16-byte reads meet all banks.
template <typename T>
constexpr int kPad = 16 / (int)sizeof(T);

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

// Two result tiles (rows 0..15 and 16..31 of a step) as one operand.
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> make_frag(f32x4 lo, f32x4 hi)
{
    Frag<T, P> f;
    f32x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    if constexpr (sizeof(T) == 4) {
        f.p[0] = x;
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            f.p[i] = __builtin_convertvector(x, bf16x8);
            if (i + 1 < P) x -= __builtin_convertvector(f.p[i], f32x8);
        }
    }
    return f;
}

// A lane's 8 values of step ks of LDS row `row` (row stride ld, planes
// `plane` elements apart).
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> load_frag(const T *base, int row, int ld, int ks, int lg, int plane)
{
    Frag<T, P> f;
    const T *a = base + row * ld + ks * 32 + lg * 8;
#pragma unroll
    for (int i = 0; i < P; ++i)
        f.p[i] = *reinterpret_cast<const typename Num<T>::Oct *>(a + i * plane);
    return f;
}

// ... of an array in fragment order.
template <typename T, int P>
__device__ __forceinline__ Frag<T, P> load_packed(const T *base, int frag, int lane)
{
    Frag<T, P> f;
#pragma unroll
    for (int i = 0; i < P; ++i)
        f.p[i] = *reinterpret_cast<const typename Num<T>::Oct *>(base + i * kFragElems + (frag * 64 + lane) * 8);
    return f;
}

// Fragments of a lower triangle: row tile `it` needs steps 0 .. it / 2; of an
// upper one (a transposed lower): steps it / 2 .. 1.
__device__ __forceinline__ constexpr int low_frag(int it, int ks) { return it < 2 ? it : 2 * it - 2 + ks; }
__device__ __forceinline__ constexpr int up_frag(int it, int ks) { return it < 2 ? 2 * it + ks : it + 2; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return (float)x; }
__device__ __forceinline__ f32x4 quad_f32(f32x4 x) { return x; }
__device__ __forceinline__ f32x4 quad_f32(bf16x4 x) { return __builtin_convertvector(x, f32x4); }

// A chunk slot's sequence, its first token (in the [B * T] token list), its
// length, and whether it is the sequence's last chunk.
struct Chunk {
    int64_t seq, tok;
    int len;
};

__device__ __forceinline__ void seq_range(const Map &m, int64_t s, int64_t &lo, int64_t &hi)
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

// The slot of a sequence's first chunk.  Packed sequence s starts at slot
// floor(start / 64) + s: ceil(len / 64) <= floor(end / 64) - floor(start / 64)
// + 1 keeps the sequences' slots apart and below T / 64 + nseq without a sum
// over the sequences before.
__device__ __forceinline__ int64_t first_slot(const Map &m, int64_t s, int64_t lo)
{
    return m.starts ? lo / kChunk + s : s * m.nck;
}

__device__ __forceinline__ Chunk locate(const Map &m, int64_t slot)
{
    Chunk c;
    int64_t lo, hi, at;
    if (!m.starts) {
        c.seq = slot / m.nck;
        seq_range(m, c.seq, lo, hi);
        at = slot - c.seq * m.nck;
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
        c.seq = a;
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
