// Host-side launch interface between the C ABI of the gated delta rule and
// the residual norm (gdr_abi.cpp) and their kernels.  Shapes and pointers
// reaching these functions are validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdr.h"
#include "residual_norm.h"

namespace wkv7 {
namespace gdr {

constexpr int kChunk = 64;   // tokens of a chunk
// A chunk's triangular factors are kept in fragment order: 6 fragments (the
// 16 x 32 blocks that touch the triangle) of 64 lanes x 8 values, per part.
constexpr int kFragElems = 6 * 64 * 8;
// bf16 parts that stand for an fp32 value as a matrix operand.
constexpr int kParts = 3;
// Per chunk and value head: 8 rows of 64 floats (gdr_prep.hip).
constexpr int kTableFloats = 8 * 64;

// Where the chunks of the sequences lie.
struct Map {
    const int32_t *starts;   // packed: [nseq + 1]; else null
    int64_t T, nseq, nck;    // tokens of a row, sequences, chunks per row (unpacked)
    int64_t slots;           // chunk slots in the workspace
};

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
    float *ws_ds = nullptr, *ws_dr = nullptr;   // [slots][Hv][K][V], [slots][Hv][64][V]
    // both
    float *table = nullptr;                     // [slots][Hv][8][64]
    void *tfrag = nullptr, *pfrag = nullptr;    // [slots][Hv][parts][6][64][8]
};

// Triangular factors and decay tables of every chunk; transposed ones for
// the backward.
hipError_t launch_prep(const Launch &a, bool transposed, hipStream_t stream);
// The forward scan over the chunks: y, sT and the record, each where asked for.
hipError_t launch_scan(const Launch &a, hipStream_t stream);
// The reverse scan: dv, ds0, and the chunks' state gradients and dR rows.
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
