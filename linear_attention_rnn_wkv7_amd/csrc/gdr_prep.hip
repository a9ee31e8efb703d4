// The triangular factors (gdr_factor.h) of every chunk and value head in
// memory, for the scans that do not make them themselves.  One wave per chunk
// and head, four to a workgroup: nothing waits at a barrier.  Bound by what it
// moves: 31 KB (bf16) written per chunk and head, 16 or 32 KB read.  Measured:
// 6560 chunks and heads, K = 128, shared keys, bf16: 81 us for 318 MB, 3.9 TB/s;
// 16384, K = 64, fp32 (21 KB written): 203 us for 898 MB, 4.4 TB/s.

#include "gdr_factor.h"

namespace wkv7 {
namespace gdr {
namespace {

template <typename T>
struct PrepArgs {
    Map map;
    const T *q, *k;
    const float *g, *beta;
    float *table;
    char *factors;
    int64_t Hk, Hv;
    int group, norm;
    float scale;
};

template <typename T, int K, bool kTrans>
__global__ void __launch_bounds__(256, 2) gdr_prep_kernel(PrepArgs<T> a)
{
    __shared__ __align__(16) FactorLds lds[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    // Workgroups go round the 8 dies; those of one die take the heads of one
    // set of chunks before the next, so that g and beta, a few bytes of each
    // line to a head, are fetched once.
    const int64_t at = blockIdx.x >> 3;
    const int64_t slot = (at / a.Hv * 8 + (blockIdx.x & 7)) * 4 + w, hv = at % a.Hv, hk = hv / a.group, ch = slot * a.Hv + hv;
    if (slot >= a.map.slots) return;
    const Chunk c = locate(a.map, slot);
    if (c.len == 0) return;
    const int64_t o = (c.tok * a.Hk + hk) * K, og = c.tok * a.Hv + hv;
    Factor<T> &to = reinterpret_cast<Factor<T> *>(a.factors)[ch];
    Factors<T, K, kTrans> f;
    f.products(lds[w], a.k + o, a.q + o, a.g + og, a.beta + og, a.Hk, a.Hv, c.len, a.norm, a.scale, lane);
    f.decays(lds[w], kTrans ? a.table + ch * kTableFloats : nullptr, c.len, lane);
    f.solve(lds[w], lane);
    f.finish(to.t, to.p, to.w, lane);
}

template <typename T, int K>
hipError_t launch_t(const Launch &a, bool transposed, hipStream_t stream)
{
    PrepArgs<T> p;
    p.map = a.map;
    p.q = static_cast<const T *>(a.q);
    p.k = static_cast<const T *>(a.k);
    p.g = a.g;
    p.beta = a.beta;
    p.table = a.table;
    p.factors = static_cast<char *>(a.factors);
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.group = (int)(a.Hv / a.Hk);
    p.norm = a.norm;
    p.scale = a.scale;
    const dim3 grid((unsigned)prep_blocks(a.map.slots, a.Hv));
    if (transposed)
        hipLaunchKernelGGL((gdr_prep_kernel<T, K, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((gdr_prep_kernel<T, K, false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

size_t factor_bytes(int dtype, bool)
{
    return dtype == WKV7_F32 ? sizeof(Factor<float>) : sizeof(Factor<bf16>);
}

hipError_t launch_prep(const Launch &a, bool transposed, hipStream_t stream)
{
    if (a.dtype == WKV7_F32)
        return a.K == 64 ? launch_t<float, 64>(a, transposed, stream) : launch_t<float, 128>(a, transposed, stream);
    return a.K == 64 ? launch_t<bf16, 64>(a, transposed, stream) : launch_t<bf16, 128>(a, transposed, stream);
}

}  // namespace gdr
}  // namespace wkv7
