// Attention of new tokens over the paged cache.
//
// Bound by the bytes of the cache: the queries of all heads that share a key
// head (and of all new tokens) go over it together, kDecodeRows to a
// workgroup, and few of them leave the matrix units idle most of the time, so
// the weights take part in two bf16 parts at no cost (over an 8-bit cache, whose
// values are rounded more coarsely, in one).  The cache of a row is cut
// into `splits` parts of whole steps; within a workgroup each wave takes
// every fourth step of the part by itself, with its own running maximum, sum
// and O^T, without a barrier: the next step's keys and values are on their
// way to registers while one is computed, and go to LDS of the wave's own.  The
// waves are joined through LDS, the parts by a second kernel, both in order.
//
// 64 rows of 8192 positions, 32 / 8 heads of 128, bf16: 285 us, 5.7 TB/s (a large
// copy: 5.2).  Over an 8-bit cache it waits for memory with too little on its way, one
// step of 4 KB a wave, half of bf16's: 2 rows of 131072, heads of 64, 39 us where the
// cache lies in the device's own, 55 to 72 from memory, 3.0 to 3.9 TB/s; its vector
// instructions are some 0.4 of the time.  In fp32 the matrix instruction bounds it, which
// takes 8 times bf16's time for 32 rows of queries however few there are: 8 bits
// under fp32 1.2 to 1.5 TB/s.  Two steps ahead, tried with heads of 128: slower, for want
// of registers.

#include <type_traits>

#include "attn_device.h"

namespace wkv7 {
namespace attn {
namespace {

template <typename T>
struct DecArgs {
    const T *q;
    const char *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    T *y;
    float *part_o;
    f32x2 *part_ml;
    int64_t T_, Hq, Hk, pages, max_pages, q_stride, rows;   // rows: T_ times group
    int group, log_page, splits;
    float scale;
};

struct E4m3 {
    uint8_t x;
};

// 16 bytes of the cache as values of T.
template <typename T, typename C>
struct Widen;
template <typename T>
struct Widen<T, T> {
    static constexpr int kPieces = 1;   // 16-byte pieces of T
    __device__ static __forceinline__ void to(f32x4 x, f32x4 (&y)[1]) { y[0] = x; }
};
template <>
struct Widen<bf16, E4m3> {
    static constexpr int kPieces = 2;
    __device__ static __forceinline__ void to(f32x4 x, f32x4 (&y)[2])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = x[i];
            const int u = __builtin_bit_cast(int, f);
            const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.f, false);
            const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.f, true);
            y[i >> 1][2 * (i & 1)] = __builtin_bit_cast(float, a);
            y[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(float, b);
        }
    }
};
template <>
struct Widen<float, E4m3> {
    static constexpr int kPieces = 4;
    __device__ static __forceinline__ void to(f32x4 x, f32x4 (&y)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = x[i];
            const int u = __builtin_bit_cast(int, f);
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(u, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(u, true);
            y[i] = f32x4{a[0], a[1], b[0], b[1]};
        }
    }
};

// The 32 tokens of a step: two halves of 16, each in one page.
template <typename T, typename C, int D>
struct Step {
    static constexpr int kBytes = 32 * D * (int)sizeof(C), kLoads = kBytes / 1024;
    static constexpr bool kE4m3 = sizeof(C) == 1;
    f32x4 k[kLoads], v[kLoads];
    float ks, vs;       // of token lane % 32
    bool there[2];      // the halves' pages

    // `n` tokens of the row from tok0 on are there.
    __device__ __forceinline__ void load(const DecArgs<T> &p, const int32_t *table, int64_t hk, int64_t tok0, int64_t n,
                                         int lane)
    {
        int64_t at[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t tok = tok0 + 16 * i;
            int page = -1;
            if (16 * i < n && (tok >> p.log_page) < p.max_pages) page = table[tok >> p.log_page];
            page = __builtin_amdgcn_readfirstlane(page);
            there[i] = page >= 0 && page < p.pages;
            at[i] = ((((there[i] ? page : 0) * p.Hk + hk) << p.log_page) + (tok & ((1 << p.log_page) - 1))) * D;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int hf = i / (kLoads / 2);
            k[i] = v[i] = gdr::zero4();
            if (there[hf]) {
                const int64_t o = at[hf] * (int64_t)sizeof(C) + (i % (kLoads / 2)) * 1024 + lane * 16;
                k[i] = *reinterpret_cast<const f32x4 *>(p.k + o);
                // what lies behind the row's end may be anything, a NaN too
                const int row = (i * 1024 + lane * 16) / (D * (int)sizeof(C));
                if (row < n) v[i] = *reinterpret_cast<const f32x4 *>(p.v + o);
            }
        }
        if (kE4m3) {
            const int hf = (lane >> 4) & 1;
            ks = vs = 0.f;
            if ((hf ? there[1] : there[0]) && (lane & 31) < n) {
                const int64_t o = (hf ? at[1] : at[0]) / D + (lane & 15);
                ks = p.k_scale[o];
                vs = p.v_scale[o];
            }
        }
    }
    // Into LDS as tiles of T.
    __device__ __forceinline__ void land(char *kt, char *vt, float *scales, int lane) const
    {
        using L = Tile<T, D>;
        using W = Widen<T, C>;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int byte = i * 1024 + lane * 16, row = byte / (D * (int)sizeof(C));
            const int piece = byte % (D * (int)sizeof(C)) / 16 * W::kPieces;
            f32x4 x[W::kPieces], y[W::kPieces];
            W::to(k[i], x);
            W::to(v[i], y);
#pragma unroll
            for (int j = 0; j < W::kPieces; ++j) {
                *reinterpret_cast<f32x4 *>(kt + L::at(row, piece + j)) = x[j];
                *reinterpret_cast<f32x4 *>(vt + L::at(row, piece + j)) = y[j];
            }
        }
        if (kE4m3 && lane < 32) {
            scales[lane] = ks;
            scales[32 + lane] = vs;
        }
    }
};

// O += the weights' products with the values: in two bf16 parts, or in one where
// the values have been rounded to 8 bits before.
template <typename T, int D, bool kParts, bool kFinite>
__device__ __forceinline__ void add_values(f32x16 (&o)[D / 32], const f32x16 &w, const Tile<T, D> &tl, const char *vt)
{
    f32x16 rest;
    if constexpr (kParts) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const uint32_t u = pack_bf16(w[i], w[i + 1]);
            rest[i] = w[i] - bf16_lo(u);
            rest[i + 1] = w[i + 1] - bf16_hi(u);
        }
    }
#pragma unroll
    for (int ss = 0; ss < 2; ++ss) {
        const Oct<T> a = as_operand<T>(w, ss);
        Oct<T> b;
        if constexpr (kParts) b = as_operand<T>(rest, ss);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) {
            Oct<T> x = tl.col(vt, dt, ss);
            if constexpr (kFinite) x = finite_of<T>(x);
            o[dt] = mma(x, a, o[dt]);
            if constexpr (kParts) o[dt] = mma(x, b, o[dt]);
        }
    }
}

// Whether a tile's 32 rows are finite (the same in all lanes).
template <typename T, int D>
__device__ __forceinline__ bool tile_finite(const char *tile, int lane)
{
    using L = Tile<T, D>;
    typedef T Piece __attribute__((ext_vector_type(16 / sizeof(T))));
    float top = 0.f;
#pragma unroll 2
    for (int n = 0; n < 32 / L::kPerCopy; ++n) {
        const Piece x = *reinterpret_cast<const Piece *>(tile + n * L::kGroup + lane * 16);
#pragma unroll
        for (int j = 0; j < 16 / (int)sizeof(T); ++j) top = __builtin_elementwise_maximum(top, __builtin_fabsf((float)x[j]));
    }
    return !__any(!(top < -kNegInf));
}

// What is not finite of the values of `n` tokens of the row from tok0 on, to the lanes
// whose columns see them: the first `here` of them.
template <typename T, typename C, int D>
__device__ __forceinline__ void add_cached(f32x16 (&o)[D / 32], const DecArgs<T> &p, const int32_t *table, int64_t hk,
                                           int64_t tok0, int n, int here, int half)
{
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int64_t tok = tok0 + j;
        const int page = __builtin_amdgcn_readfirstlane(table[tok >> p.log_page]);
        if (page < 0 || page >= p.pages) continue;
        const int64_t row = ((page * p.Hk + hk) << p.log_page) + (tok & ((1 << p.log_page) - 1));
        if constexpr (sizeof(C) == sizeof(T)) {
            add_odd<T, D, false>(o, reinterpret_cast<const T *>(p.v) + row * D, 0, 1, j < here ? 1 : 0, half);
        } else {
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(p.v + row * D + 32 * dt + reg_row(i, half));
#pragma unroll
                    for (int m = 0; m < 4; ++m)   // e4m3 has NaN, and no infinity
                        if (j < here && (u >> 8 * m & 0x7f) == 0x7f) o[dt][i + m] += __builtin_nanf("");
                }
        }
    }
}

// A token that has seen nothing has 0.
__device__ __forceinline__ f32x4 quotient(f32x4 x, float sum)
{
    return sum == 0.f ? gdr::zero4() : x * (1.f / sum);
}

// Waves on a SIMD that the registers are divided for.  2 rows of 131072 tokens, 4 new
// ones, 32 / 8 heads, bf16, one and two: heads of 64 109 and 119 us, of 128 206 and
// 196, in 8 bits 80 and 81, 228 and 139.
template <typename T, int D>
constexpr int kDecodeOccupancy = sizeof(T) == 2 ? (D == 64 ? 1 : 2) : (D == 64 ? 2 : 1);

// kMany: several new tokens to a row, of which the earlier ones do not see the later
// ones' values.  The few steps where they differ run in a loop of their own, which costs
// nothing (4 tokens over 131072, heads of 64, in 8 bits 57 and 56 us, in bf16 97 and 98);
// the kernel for single tokens is without it.
template <typename T, typename C, int D, bool kMany>
__global__ void __launch_bounds__(256, (kDecodeOccupancy<T, D>)) attn_decode_kernel(DecArgs<T> p)
{
    using L = Tile<T, D>;
    using S = Step<T, C, D>;
    constexpr int kTileBytes = L::bytes(kDecodeStep);
    // a wave's tiles; then, of each wave, O by rows
    constexpr int kOut = kDecodeRows * (D + 4) * 4;
    constexpr int kWave = 2 * kTileBytes > kOut ? 2 * kTileBytes : kOut;
    __shared__ __attribute__((aligned(16))) char lds[4][kWave];
    __shared__ __attribute__((aligned(16))) float scales[4][64];
    __shared__ float stat[4][2][kDecodeRows];   // maximum, sum
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, l32 = lane & 31;
    L tl;
    tl.init(lane);
    const int64_t tiles = (p.rows + kDecodeRows - 1) / kDecodeRows;
    const int64_t hk = blockIdx.y / tiles, tile = blockIdx.y - hk * tiles, b = blockIdx.z;
    const int split = blockIdx.x;

    const int64_t past = p.lens[b] - p.T_, most = p.max_pages << p.log_page;
    // a token sees `sees` positions, the tile's first and last `all` and `len` of them;
    // those past the table hold nothing
    const int64_t r = tile * kDecodeRows + l32;
    const int64_t t = r / p.group, hq = hk * p.group + (r - t * p.group);
    const bool live = r < p.rows;
    const int64_t sees = live ? past + t + 1 : 0;
    const int64_t end = (tile + 1) * kDecodeRows < p.rows ? (tile + 1) * kDecodeRows : p.rows;
    const int64_t all = past + tile * kDecodeRows / p.group + 1;
    int64_t len = past + (end - 1) / p.group + 1;
    len = len < 0 ? 0 : len < most ? len : most;
    const int64_t steps = (len + kDecodeStep - 1) / kDecodeStep, per = (steps + p.splits - 1) / p.splits;
    const int64_t last = (split + 1) * per < steps ? (split + 1) * per : steps;

    Oct<T> q[D / 16];
    {
        const T *qp = p.q + (b * p.T_ + t) * p.q_stride + hq * D + 8 * half;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            q[ks] = zero_oct<T>();
            if (live) q[ks] = *reinterpret_cast<const Oct<T> *>(qp + 16 * ks);
        }
    }
    f32x16 o[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();
    float ref = kLowest, l = 0.f;   // ref: the maximum times c
    const float c = p.scale * kLog2e;
    char *kt = lds[wave], *vt = kt + kTileBytes;
    const int32_t *table = p.table + b * p.max_pages;

    S next;
    const int64_t begin = split * per + wave;
    if (begin < last) next.load(p, table, hk, begin * kDecodeStep, len - begin * kDecodeStep, lane);
    bool odd = false;   // whether something was left out
    auto step = [&](int64_t at, auto cut) __attribute__((always_inline)) {
        constexpr bool kCut = decltype(cut)::value;
        next.land(kt, vt, scales[wave], lane);
        const bool there0 = next.there[0], there1 = next.there[1];
        if (at + 4 < last) next.load(p, table, hk, (at + 4) * kDecodeStep, len - (at + 4) * kDecodeStep, lane);
        gdr::wave_sync();
        f32x16 s = zero16();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) s = mma(tl.row(kt, ks), q[ks], s);
        if (S::kE4m3) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&scales[wave][reg_row(i, half)]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i + j] *= x[j];
            }
        }
        // Where some token sees not all of the step.  (The empty asm keeps the branch: as
        // selects this would be done in every step.)
        if (!(there0 && there1 && (at + 1) * kDecodeStep <= len && (at + 1) * kDecodeStep <= all)) {
            asm volatile("");
            const int64_t seen = sees - at * kDecodeStep;
            const int here = seen < 0 ? 0 : seen < kDecodeStep ? (int)seen : kDecodeStep;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (reg_row(i, half) >= here || !(i < 8 ? there0 : there1)) s[i] = kNegInf;
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top = half_max(top) * c;
        // a row keeps its reference until its maximum is 2^8 times what that stands for
        const bool grown = top > ref + 8.f;
        if (__any(grown)) {
            asm volatile("");
            const float to = grown ? top : ref, alpha = __builtin_amdgcn_exp2f(grown ? ref - to : 0.f);
            ref = to;
            l *= alpha;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= alpha;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -ref));
            sum += s[i];
        }
        l += sum;
        if (S::kE4m3) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&scales[wave][32 + reg_row(i, half)]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i + j] *= x[j];
            }
        }
        if (kCut) {
            const int64_t seen = sees - at * kDecodeStep;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (reg_row(i, half) >= seen) s[i] = 0.f;   // also times a scale that is NaN
            odd = odd || !tile_finite<T, D>(vt, lane);
        }
        add_values<T, D, sizeof(T) == 2 && !S::kE4m3, kCut>(o, s, tl, vt);
        gdr::wave_sync();
    };
    int64_t at = begin;
    for (; at < last && (!kMany || (at + 1) * kDecodeStep <= all || all == len); at += 4) step(at, std::false_type{});
    if constexpr (kMany) {
        // Steps that the mask cuts through, one or two of the tile's: what is not finite of
        // the values stays out, and the tokens that see it get it behind the last step.
        const int64_t cut = at;
#pragma unroll 1
        for (; at < last; at += 4) step(at, std::true_type{});
        if (odd)
            for (at = cut; at < last; at += 4) {
                const int64_t n = len - at * kDecodeStep, seen = sees - at * kDecodeStep;
                add_cached<T, C, D>(o, p, table, hk, at * kDecodeStep, n < kDecodeStep ? (int)n : kDecodeStep,
                                    seen < 0 ? 0 : seen < kDecodeStep ? (int)seen : kDecodeStep, half);
            }
    }

    // the four waves
    l = half_sum(l);
    if (half == 0) {
        stat[wave][0][l32] = ref;
        stat[wave][1][l32] = l;
    }
    put_rows<D>(lds[wave], o, lane);
    __syncthreads();
    constexpr int kLanes = D / 4;   // of a row
    for (int i = threadIdx.x / kLanes; i < kDecodeRows; i += 256 / kLanes) {
        const int64_t row = tile * kDecodeRows + i;
        if (row >= p.rows) break;
        const int col = 4 * (threadIdx.x % kLanes);
        float top = kLowest, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[w][0][i]);
        f32x4 x = gdr::zero4();
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float a = __builtin_amdgcn_exp2f(stat[w][0][i] - top);
            sum += a * stat[w][1][i];
            x += a * get_row<D>(lds[w], i, col);
        }
        const int64_t tt = row / p.group, to = (b * p.T_ + tt) * p.Hq + hk * p.group + (row - tt * p.group);
        if (p.part_o) {
            *reinterpret_cast<f32x4 *>(p.part_o + (to * p.splits + split) * D + col) = x;
            if (col == 0) p.part_ml[to * p.splits + split] = f32x2{top, sum};
        } else {
            *reinterpret_cast<Quad<T> *>(p.y + to * D + col) = __builtin_convertvector(quotient(x, sum), Quad<T>);
        }
    }
}

// The parts of a row: a workgroup to a row, D / 4 lanes to a part, every
// 256 / (D / 4)th of them to the same lanes; then those, in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const float *part_o, const f32x2 *part_ml, T *y, int64_t rows,
                                                        int splits)
{
    constexpr int L = D / 4, G = 256 / L;
    __shared__ __attribute__((aligned(16))) f32x4 red[G][L];
    __shared__ float tops[G], sums[G];
    const int lane = threadIdx.x % L, g = threadIdx.x / L;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const f32x2 *ml = part_ml + row * splits;
        const float *po = part_o + row * splits * D + 4 * lane;
        float top = kLowest, sum = 0.f;
        f32x4 x = gdr::zero4();
        for (int s = g; s < splits; s += G) top = fmaxf(top, ml[s][0]);
        for (int s = g; s < splits; s += G) {
            const f32x2 st = ml[s];
            const float a = __builtin_amdgcn_exp2f(st[0] - top);
            sum += a * st[1];
            x += a * *reinterpret_cast<const f32x4 *>(po + (int64_t)s * D);
        }
        red[g][lane] = x;
        if (lane == 0) {
            tops[g] = top;
            sums[g] = sum;
        }
        __syncthreads();
        if (g == 0) {
            top = kLowest;
#pragma unroll
            for (int i = 0; i < G; ++i) top = fmaxf(top, tops[i]);
            sum = 0.f;
            x = gdr::zero4();
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float a = __builtin_amdgcn_exp2f(tops[i] - top);
                sum += a * sums[i];
                x += a * red[i][lane];
            }
            *reinterpret_cast<Quad<T> *>(y + row * D + 4 * lane) = __builtin_convertvector(quotient(x, sum), Quad<T>);
        }
        __syncthreads();
    }
}

template <typename T, typename C, int D>
hipError_t launch_t(const DecodeLaunch &a, hipStream_t stream)
{
    DecArgs<T> p;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const char *>(a.k_pages);
    p.v = static_cast<const char *>(a.v_pages);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.table = a.table;
    p.lens = a.lens;
    p.y = static_cast<T *>(a.y);
    p.part_o = a.part_o;
    p.part_ml = reinterpret_cast<f32x2 *>(a.part_ml);
    p.T_ = a.T;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.pages = a.pages;
    p.max_pages = a.max_pages;
    p.q_stride = a.q_stride;
    p.group = (int)(a.Hq / a.Hk);
    p.rows = a.T * p.group;
    p.log_page = __builtin_ctzll((unsigned long long)a.page);
    p.splits = (int)a.splits;
    p.scale = a.scale;
    const int64_t tiles = (p.rows + kDecodeRows - 1) / kDecodeRows;
    const dim3 grid((unsigned)a.splits, (unsigned)(a.Hk * tiles), (unsigned)a.B);
    if (a.T > 1)
        hipLaunchKernelGGL((attn_decode_kernel<T, C, D, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((attn_decode_kernel<T, C, D, false>), grid, dim3(256), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = a.B * a.T * a.Hq;
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(grid_of(rows)), dim3(256), 0, stream,
                       p.part_o, p.part_ml, p.y, rows, p.splits);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const DecodeLaunch &a, hipStream_t stream)
{
    if (a.cache_dtype == KV_CACHE_E4M3)
        return a.D == 64 ? launch_t<T, E4m3, 64>(a, stream) : launch_t<T, E4m3, 128>(a, stream);
    return a.D == 64 ? launch_t<T, T, 64>(a, stream) : launch_t<T, T, 128>(a, stream);
}

}  // namespace

hipError_t launch_decode(const DecodeLaunch &a, hipStream_t stream)
{
    return a.dtype == WKV7_F32 ? launch_d<float>(a, stream) : launch_d<bf16>(a, stream);
}

}  // namespace attn
}  // namespace wkv7
