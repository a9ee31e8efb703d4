// Host-side launch interface between the C ABI of the gated delta rule and
// the residual norm (gdr_abi.cpp) and their kernels.  Shapes and pointers
// reaching these functions are validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "gdr.h"
#include "residual_norm.h"

namespace wkv7 {
namespace gdr {

constexpr int kChunk = 64;   // tokens of a chunk
// bf16 parts that stand for an fp32 value as a matrix operand.
constexpr int kParts = 3;
// Per chunk and value head, from the reverse scan to the gradients, per
// token: the inclusive sum of g log2(e) as a sum of two floats, beta, and the
// reciprocal lengths of k and (times the scale) q.
constexpr int kTableFloats = 5 * 64;

// Where the chunks of the sequences lie.  Rows that are not packed may be cut
// into nseg segments of nckseg chunks; the scans take those as sequences.
struct Map {
    const int32_t *starts;   // packed: [nseq + 1]; else null
    int64_t T, nseq, nck;    // tokens of a row, sequences, chunks per row (unpacked)
    int64_t slots;           // chunk slots in the workspace
    int64_t nseg, nckseg;
};

// Whether the scans' workgroups make the chunks' triangular factors themselves
// (gdr_scan.hip) or find them in memory, made by a kernel before (gdr_prep.hip).
// In memory they cost 31 KB per chunk and head, written and read, against 32 KB
// of inputs and outputs at K = V = 64 in bf16: there calls take, made here
// against made before, 248 us against 404 (8 x 4096 x 32, forward) and 812 against
// 982 (backward).  With V = 128 each of a head's two workgroups makes them: 473
// and 482 us.  In fp32 the making of a chunk's factors takes longer than its slabs
// do: 750 and 550.  With K = 128 there is no room in LDS.  Below 128 heads in
// flight it gains little (1 x 960 x 32: 53 and 57 us), and long rows run in
// segments, which read the factors twice.  Packed sequences count as heads in
// flight whatever their lengths, which only the device knows (x 32 heads, 24 of
// 12288 tokens together: 136 and 187 us; 8 of 32768: 322 and 445); where most of
// them are shorter than a chunk the factors are better made before (300 of 40
// tokens: 412 and 320; one of 12288 beside 40 of one: 702 and 607).
inline bool scan_makes_factors(int dtype, int64_t K, int64_t V, int64_t units)
{
    return dtype == WKV7_BF16 && K == 64 && V <= 64 && units >= 128;
}
// Waves that make them.
constexpr int kMakers = 4;

// The grid of a scan.  Slabs of 16 columns per workgroup, a wave each: as many
// as there are (8 at most, 4 beside makers), fewer while that leaves compute
// units without a workgroup.  A unit's slab groups read the same q, k and
// factors, a key head's value heads the same q and k: they go to one die, whose
// cache then holds them for all, unless that leaves a die with more than an
// eighth above its share and its 32 compute units.  (4 x 4096 x 8 / 16 heads, K =
// V = 128, bf16, four groups, apart and together: forward 332 and 314 us, reverse
// 305 and 291; with one group to a head it makes no difference: 24 packed sequences
// of 12288 tokens, 16 / 32 heads, 224 and 222.)
struct ScanGrid {
    int64_t slabs;                  // of a workgroup
    int64_t groups, share, total;   // slab groups of a unit, neighbours on a die, workgroups with work
    int64_t blocks, threads;        // of the launch
};
inline ScanGrid scan_grid(int64_t units, int64_t heads_per_key, int64_t columns, bool makes)
{
    ScanGrid g;
    const int64_t slabs = columns / 16, most = makes ? 4 : 8;
    g.groups = (slabs + most - 1) / most;
    while (units * g.groups < 256 && g.groups < slabs) ++g.groups;
    g.slabs = (slabs + g.groups - 1) / g.groups;
    g.groups = (slabs + g.slabs - 1) / g.slabs;
    g.total = units * g.groups;
    int64_t turns = 0;
    for (int64_t s : {g.groups * heads_per_key, g.groups, (int64_t)1}) {
        g.share = s;
        turns = (g.total / s + 7) / 8 * s;   // a die's most
        if (turns <= 32 || turns * 64 <= g.total * 9) break;
    }
    g.blocks = turns * 8;
    g.threads = 64 * (g.slabs + (makes ? kMakers : 1));
    return g;
}
// Workgroups of the factors' (256 threads) and the gradients' kernel (4 K).
inline int64_t prep_blocks(int64_t slots, int64_t Hv) { return (slots + 31) / 32 * 8 * Hv; }
inline int64_t grads_blocks(int64_t slots, int64_t Hk) { return (slots + 7) / 8 * 8 * Hk; }

// Bytes of a chunk's factors in memory, for the forward or (transposed) the reverse scan.
size_t factor_bytes(int dtype, bool transposed);

struct Launch {
    Map map;
    int64_t B, Hk, Hv, K, V;
    int dtype, norm;
    float scale;
    const void *q = nullptr, *k = nullptr, *v = nullptr;
    const float *g = nullptr, *beta = nullptr, *s0 = nullptr;
    void *y = nullptr;
    float *sT = nullptr;
    float *rec_s = nullptr, *rec_e = nullptr;   // the record, or null
    // backward
    const void *dy = nullptr;
    const float *dsT = nullptr;
    void *dq = nullptr, *dk = nullptr, *dv = nullptr;
    float *dg = nullptr, *dbeta = nullptr, *ds0 = nullptr;
    float *ws_ds = nullptr, *ws_dr = nullptr;   // [slots][Hv][V][K], [slots][Hv][64][V]
    float *table = nullptr;                     // [slots][Hv][5][64]
    void *factors = nullptr;                    // [slots][Hv][factor_bytes], or null
    // segments: how each takes its state on, and the states they start from
    float *seg_map = nullptr;                   // [nseq * nseg][Hv][K][V + K]
    float *carry = nullptr;                     // [nseq * nseg][Hv][V][K]
};

// The factors of every chunk; transposed ones, and the tables, for the backward.
hipError_t launch_prep(const Launch &a, bool transposed, hipStream_t stream);
// The forward scan over the chunks: y, sT and the record, each where asked for.
hipError_t launch_scan(const Launch &a, hipStream_t stream);
// The reverse scan: dv, ds0, and the chunks' state gradients, dR rows and tables.
hipError_t launch_reverse(const Launch &a, hipStream_t stream);
// dq, dk, dg, dbeta of every chunk.
hipError_t launch_grads(const Launch &a, hipStream_t stream);

struct DecodeLaunch {
    int64_t B, T, Hk, Hv, K, V, pool;
    int dtype, norm;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    void *y;
};
hipError_t launch_decode(const DecodeLaunch &a, hipStream_t stream);

struct EpilogueLaunch {
    int64_t rows, H, N, Hw;
    int dtype;
    float eps;
    const void *y, *gate, *dz = nullptr;
    const float *w;
    void *z = nullptr, *dy = nullptr, *dgate = nullptr;
    float *dw = nullptr, *part = nullptr;
};
// Backward workgroups per weight head (each a range of rows).
int64_t epilogue_parts(int64_t rows, int64_t H, int64_t N, int64_t Hw);
hipError_t launch_epilogue_forward(const EpilogueLaunch &a, hipStream_t stream);
hipError_t launch_epilogue_backward(const EpilogueLaunch &a, hipStream_t stream);

struct NormLaunch {
    int64_t rows, D;
    int dtype;
    float eps;
    const void *x = nullptr, *y = nullptr, *dh = nullptr, *dx_out = nullptr;
    const float *scale = nullptr, *w = nullptr;
    void *x_out = nullptr, *h = nullptr, *dx = nullptr, *dy = nullptr;
    float *dw = nullptr, *dscale = nullptr, *part = nullptr;
};
// Backward workgroups (each a range of rows).
int64_t norm_parts(int64_t rows, int64_t D);
hipError_t launch_norm_forward(const NormLaunch &a, hipStream_t stream);
hipError_t launch_norm_backward(const NormLaunch &a, hipStream_t stream);

}  // namespace gdr
}  // namespace wkv7
