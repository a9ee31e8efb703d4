// The paged cache of keys and values: new tokens into their pages, as they are
// or in 8 bits, and sequences back out of them.
//
// Both are bound by memory: D / 8 lanes to a token's head, 8 entries to a lane,
// one pass.  The scale of a head in 8 bits is max|x| times the fp32 number
// nearest to 1 / 448, and x is divided by it in correctly rounded fp32, so that
// a stored value depends on nothing but its head.
//
// 32768 packed tokens, 8 heads of 128, bf16 to 8 bits: write 57 us (3.6 TB/s), read
// back 37 (5.5).  The write has 378 vector instructions a wave, most of them for the
// quotients; with the compiler's division, and each load after the last store, it
// took 74 us, the read 43.

#include "attn_device.h"

namespace wkv7 {
namespace attn {
namespace {

constexpr float kE4m3Max = 448.f;

template <typename T>
struct CacheArgs {
    const T *k, *v;
    T *k_out, *v_out;
    const char *kp, *vp;
    char *kp_out, *vp_out;
    float *ks, *vs;
    const int32_t *table, *lens, *starts;
    int64_t rows, T_, Hk, pages, max_pages, k_stride, v_stride, tokens;
    int log_page, small;
};

// Where a token lies: its page, and its place there, if it has one; owned: whether
// it is a row's at all.  L lanes look for one token.
template <int L, typename T>
__device__ __forceinline__ bool find(const CacheArgs<T> &a, uint32_t tok, int &page, int &offset, bool &owned)
{
    int r, i, n;
    if (!a.starts) {
        r = (int)(tok / (uint32_t)a.T_);
        i = (int)(tok - (uint32_t)r * (uint32_t)a.T_);
        n = (int)a.T_;
    } else {
        // the last row that starts at or before it: each lane asks at one place of the range
        const int lane = threadIdx.x % L, shift = (threadIdx.x & 63) / L * L;
        int step = 1;
        while ((int64_t)step * L < a.rows) step *= L;
        for (r = 0; step; step /= L) {
            const int64_t s = r + (int64_t)lane * step;
            const bool before = s < a.rows && a.starts[s] <= (int)tok;
            const int count = __popcll(__ballot(before) >> shift & ((1ull << L) - 1));
            r += (count > 0 ? count - 1 : 0) * step;
        }
        const int all = (int)a.tokens;
        int b = a.starts[r], e = a.starts[r + 1];
        b = b < 0 ? 0 : b > all ? all : b;
        e = e < b ? b : e > all ? all : e;
        i = (int)tok - b;
        n = e - b;
    }
    owned = i >= 0 && i < n;
    if (!owned) return false;
    const int64_t pos = (int64_t)a.lens[r] - n + i;
    if (pos < 0 || (pos >> a.log_page) >= a.max_pages) return false;
    page = a.table[r * a.max_pages + (pos >> a.log_page)];
    offset = (int)pos & ((1 << a.log_page) - 1);
    return page >= 0 && page < a.pages;
}

// x / by, correctly rounded.  r is 1 / by, correctly rounded, and the first quotient
// is off by less than two units in the last place; each step adds the exact rest's
// share, after which the quotient is off by less than one, and then rounded as it
// should be (Markstein), unless by is one of the numbers whose last bits are all
// set or the rest leaves the normal range: those are divided.
struct Divide {
    float by, r;
    bool plain;
    __device__ __forceinline__ explicit Divide(float b) : by(b), r(1.f / b)
    {
        const uint32_t u = __builtin_bit_cast(uint32_t, b);
        plain = !(b > 0x1p-60f && b < 0x1p60f) || (u & 0x7fffff) == 0x7fffff;
    }
    __device__ __forceinline__ float operator()(float x) const
    {
        float q = x * r;
        q = fmaf(fmaf(-q, by, x), r, q);
        return fmaf(fmaf(-q, by, x), r, q);
    }
};

template <int L>
__device__ __forceinline__ float lanes_max(float x)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

template <typename T>
__device__ __forceinline__ f32x8 wide(Oct<T> x)
{
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __builtin_convertvector(x, f32x8);
}

template <typename T, int D, bool kE4m3>
__device__ __forceinline__ void put(Oct<T> src, char *pages, float *scales, int64_t row, int col)
{
    if constexpr (!kE4m3) {
        *reinterpret_cast<Oct<T> *>(pages + (row * D + col) * (int64_t)sizeof(T)) = src;
    } else {
        const f32x8 x = wide<T>(src);
        float top = 0.f, odd = 0.f;   // odd: NaN with an infinity or NaN among x, or 0
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top = fmaxf(top, fabsf(x[j]));
            odd += x[j] * 0.f;
        }
        top = lanes_max<D / 8>(top);
#pragma unroll
        for (int d = 1; d < D / 8; d <<= 1) odd += __shfl_xor(odd, d);
        const float scale = top * (1.f / kE4m3Max) + odd, by = scale > 0.f ? scale : 1.f;
        float z[8];
        const Divide divide(by);
        if (divide.plain) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = x[j] / by;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = divide(x[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = fminf(fmaxf(z[j], -kE4m3Max), kE4m3Max);
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], hi, true);
        *reinterpret_cast<int2 *>(pages + row * D + col) = make_int2(lo, hi);
        if (col == 0) scales[row] = scale;
    }
}

template <typename T, int D, bool kE4m3>
__device__ __forceinline__ void get(T *dst, const char *pages, const float *scales, int64_t row, int col, bool there)
{
    Oct<T> x = zero_oct<T>();
    if (there) {
        if constexpr (!kE4m3) {
            x = *reinterpret_cast<const Oct<T> *>(pages + (row * D + col) * (int64_t)sizeof(T));
        } else {
            const int2 u = *reinterpret_cast<const int2 *>(pages + row * D + col);
            const float s = scales[row];
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(u.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(u.x, true);
            const auto c = __builtin_amdgcn_cvt_pk_f32_fp8(u.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(u.y, true);
            const f32x8 z = f32x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]} * s;
            x = __builtin_convertvector(z, Oct<T>);
        }
    }
    *reinterpret_cast<Oct<T> *>(dst) = x;
}

template <typename T, int D, bool kE4m3, bool kWrite>
__global__ void __launch_bounds__(256) kv_kernel(CacheArgs<T> a)
{
    constexpr int L = D / 8;
    const int col = 8 * (threadIdx.x % L);
    for (int64_t id = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; id < a.tokens * a.Hk;   // whole heads
         id += (int64_t)gridDim.x * (256 / L)) {
        uint32_t tok;
        if (a.small)   // 32 bits hold every index of a token's head
            tok = (uint32_t)id / (uint32_t)a.Hk;
        else
            tok = (uint32_t)(id / a.Hk);
        const int64_t h = id - tok * a.Hk;
        Oct<T> k, v;   // on their way while the place is looked for
        if constexpr (kWrite) {
            k = *reinterpret_cast<const Oct<T> *>(a.k + tok * a.k_stride + h * D + col);
            v = *reinterpret_cast<const Oct<T> *>(a.v + tok * a.v_stride + h * D + col);
        }
        int page = 0, offset = 0;
        bool owned;
        const bool there = find<L>(a, tok, page, offset, owned);
        const int64_t row = ((page * a.Hk + h) << a.log_page) + offset;
        if constexpr (kWrite) {
            if (!there) continue;
            put<T, D, kE4m3>(k, a.kp_out, a.ks, row, col);
            put<T, D, kE4m3>(v, a.vp_out, a.vs, row, col);
        } else {
            if (!owned) continue;
            get<T, D, kE4m3>(a.k_out + id * D + col, a.kp, a.ks, row, col, there);
            get<T, D, kE4m3>(a.v_out + id * D + col, a.vp, a.vs, row, col, there);
        }
    }
}

template <typename T, int D, bool kE4m3>
hipError_t launch_t(const CacheLaunch &a, bool write, hipStream_t stream)
{
    CacheArgs<T> p;
    p.k = static_cast<const T *>(a.k);
    p.v = static_cast<const T *>(a.v);
    p.k_out = static_cast<T *>(a.k_out);
    p.v_out = static_cast<T *>(a.v_out);
    p.kp = static_cast<const char *>(a.k_pages);
    p.vp = static_cast<const char *>(a.v_pages);
    p.kp_out = static_cast<char *>(a.k_out);
    p.vp_out = static_cast<char *>(a.v_out);
    p.ks = a.k_scale;
    p.vs = a.v_scale;
    p.table = a.table;
    p.lens = a.lens;
    p.starts = a.starts;
    p.rows = a.rows;
    p.T_ = a.T;
    p.Hk = a.Hk;
    p.pages = a.pages;
    p.max_pages = a.max_pages;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.tokens = a.tokens;
    p.log_page = __builtin_ctzll((unsigned long long)a.page);
    p.small = a.tokens * a.Hk < (int64_t(1) << 32);
    const int64_t per = 256 / (D / 8);
    const dim3 grid(grid_of((a.tokens * a.Hk + per - 1) / per));
    if (write)
        hipLaunchKernelGGL((kv_kernel<T, D, kE4m3, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((kv_kernel<T, D, kE4m3, false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const CacheLaunch &a, bool write, hipStream_t stream)
{
    if (a.cache_dtype == KV_CACHE_E4M3)
        return a.D == 64 ? launch_t<T, 64, true>(a, write, stream) : launch_t<T, 128, true>(a, write, stream);
    return a.D == 64 ? launch_t<T, 64, false>(a, write, stream) : launch_t<T, 128, false>(a, write, stream);
}

}  // namespace

hipError_t launch_kv_write(const CacheLaunch &a, hipStream_t stream)
{
    return a.dtype == WKV7_F32 ? launch_d<float>(a, true, stream) : launch_d<bf16>(a, true, stream);
}
hipError_t launch_kv_read(const CacheLaunch &a, hipStream_t stream)
{
    return a.dtype == WKV7_F32 ? launch_d<float>(a, false, stream) : launch_d<bf16>(a, false, stream);
}

}  // namespace attn
}  // namespace wkv7
