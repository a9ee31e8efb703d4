// Host-side launch interface between the C ABI of softmax attention
// (attn_abi.cpp) and its kernels.  Shapes and pointers reaching these
// functions are validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attention.h"

namespace wkv7 {
namespace attn {

// Rows of queries (or keys, in the gradients of k and v) of a workgroup.
constexpr int kTile = 128;

// Where the tiles of the sequences lie.
struct Seqs {
    const int32_t *starts;   // packed: [nseq + 1]; else null
    int64_t T, nseq;         // tokens of a row; sequences
    int64_t tiles;           // of a row (unpacked)
    int64_t slots;           // tile slots: rows' tiles, or, packed, an upper bound of them
};

// Workgroups of a launch whose kernel goes on by the grid where `needed` are more.
inline unsigned grid_of(int64_t needed) { return (unsigned)(needed < (1 << 20) ? needed : 1 << 20); }

// Whether a launch of so many workgroups of kTile rows takes the narrow form
// instead (narrow).  Forward and backward, us, wide and narrow: bf16, 1 x
// 2048 x 8 heads of 64 (128 workgroups) 29 and 19, 81 and 48; x 16 (256) 30 and 27,
// 83 and 85; of 128: 43 and 33, 129 and 80; 48 and 63, 140 and 156.  fp32, x 16 of 64
// (256) 149 and 106, 505 and 325; of 128 270 and 186, 907 and 628; 4 x 512 x 32 (512)
// of 64 59 and 79; 1 x 4096 x 16 (512) 405 and 393.
inline bool is_narrow(int64_t workgroups, int dtype) { return workgroups < (dtype == WKV7_F32 ? 512 : 256); }

// Block -> (slot, head).  Of a unit (row, head), the tiles that have the most to go
// over start first.  Workgroups go to the 8 dies in turn: each die has units of its
// own, neighbours, and takes `chunk` of them at a time, tile by tile, so that its
// cache holds what these read.
__host__ __device__ inline void unit_of(const Seqs &m, int64_t B, int64_t heads_, uint32_t chunk, bool last_first,
                                        uint32_t id, int &slot, int &head)
{
    const uint32_t heads = (uint32_t)heads_, units = m.starts ? heads : (uint32_t)(B * heads_);
    const uint32_t tiles = (uint32_t)(m.starts ? m.slots : m.tiles);
    uint32_t tile, u;
    if (units % 8 == 0) {
        const uint32_t per = units / 8, n = id / 8, c = n / (tiles * chunk), first = c * chunk;
        const uint32_t here = per - first < chunk ? per - first : chunk, rest = n - first * tiles;
        tile = rest / here;
        u = id % 8 * per + first + (rest - tile * here);
    } else {
        tile = id / units;
        u = id - tile * units;
    }
    if (last_first) tile = tiles - 1 - tile;
    const uint32_t b = u / heads;
    head = (int)(u - b * heads);
    slot = (int)(m.starts ? tile : b * (uint32_t)m.tiles + tile);
}

// Units of a die's that are taken at a time, where `sharing` of them read the same
// `bytes`: as many as read 8 MB, twice a die's cache, and keep its compute units
// busy.  8 x 4096 x 32 heads of 64, us, forward, dq, dk and dv: all at a time (10
// times the bytes from memory) 744, 857, 1135; 2 MB 668, 833, 1085; 4 MB 675, 829,
// 1066; 8 MB 670, 821, 1059.  With 128 workgroups or fewer to a die, the order of
// their lengths counts: dk and dv of 4 x 4096 x 16 / 4 heads of 128 680, and 711 by
// units.
inline uint32_t chunk_of(const Seqs &m, int64_t units, int64_t bytes, int64_t sharing)
{
    if (m.starts || units < 8) return (uint32_t)(units < 8 ? 1 : units / 8);
    int64_t n = bytes < (8 << 20) ? (8 << 20) / bytes * sharing : sharing;
    if (n * m.tiles < 128) n = (127 + m.tiles) / m.tiles;
    return (uint32_t)(n < units / 8 ? n : units / 8);
}

// Where few workgroups of kTile rows would leave compute units without one, a
// workgroup has kNarrow rows and its four waves share what they have to go over.
constexpr int kNarrow = 32;
inline Seqs narrow(const Seqs &s, int64_t B)
{
    Seqs n = s;
    n.tiles = (s.T + kNarrow - 1) / kNarrow;
    n.slots = s.starts ? s.T / kNarrow + s.nseq : B * n.tiles;
    return n;
}

struct Launch {
    Seqs seqs;
    int64_t B, Hq, Hk, D;
    int64_t q_stride, k_stride, v_stride;   // elements
    int dtype;
    float scale;
    const void *q = nullptr, *k = nullptr, *v = nullptr;
    void *y = nullptr;
    float *lse = nullptr;
    void *record = nullptr;
    // backward
    const void *dy = nullptr;
    void *dq = nullptr, *dk = nullptr, *dv = nullptr;
    float *stats = nullptr;   // [Hq][B T][2]
};

hipError_t launch_forward(const Launch &a, hipStream_t stream);
hipError_t launch_backward(const Launch &a, hipStream_t stream);

struct QkNormLaunch {
    int64_t B, T, Hq, Hk, D, R, q_stride, k_stride;
    int dtype, interleaved;
    float eps;
    const void *q = nullptr, *k = nullptr;
    const float *wq = nullptr, *wk = nullptr, *theta = nullptr;
    const int32_t *positions = nullptr;
    void *qz = nullptr, *kz = nullptr;   // forward: out
    const void *dqz = nullptr, *dkz = nullptr;
    void *dq = nullptr, *dk = nullptr;
    float *dwq = nullptr, *dwk = nullptr, *part = nullptr;
};
// Workgroups of a launch over so many tokens (each a range of them).
inline int64_t qk_norm_parts(int64_t tokens) { return tokens < 1024 ? tokens : 1024; }
hipError_t launch_qk_norm_forward(const QkNormLaunch &a, hipStream_t stream);
hipError_t launch_qk_norm_backward(const QkNormLaunch &a, hipStream_t stream);

struct CacheLaunch {
    int64_t rows, T, Hk, D, pages, page, max_pages, k_stride, v_stride;
    int64_t tokens;   // of k and v in all
    int dtype, cache_dtype;
    const void *k, *v;
    void *k_out, *v_out;
    const void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    const int32_t *table, *lens, *starts;
};
hipError_t launch_kv_write(const CacheLaunch &a, hipStream_t stream);   // k, v -> k_out, v_out (pages)
hipError_t launch_kv_read(const CacheLaunch &a, hipStream_t stream);    // pages -> k_out, v_out

struct DecodeLaunch {
    int64_t B, T, Hq, Hk, D, pages, page, max_pages, q_stride;
    int64_t splits;
    int dtype, cache_dtype;
    float scale;
    const void *q, *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    void *y;
    float *part_o, *part_ml;   // [B T Hq][splits][D] and [..][2], or null with one split
};
// Rows of queries that share a key head's pass over the cache.
constexpr int kDecodeRows = 32;
// Tokens of a wave's step.
constexpr int kDecodeStep = 32;
// Parts of the cache that are read at once: enough for two workgroups to a compute
// unit, which it holds at a time, and of a table's full rows none under 8 steps (of
// which each wave has two).
// 256, 512, 768 and 1024 workgroups, us, bf16: 2 rows of 131072 positions, 4 new
// tokens, 32 / 8 heads of 64, 132, 103, 123, 105 (in 8 bits 122, 81, 102, 86); 16 of
// 4096, 16 / 4 heads of 128, 33, 31, 36, 34.  At least 4, 8 or 16 steps: the same.
// A row that fills less of its table is cut into as many parts, of fewer steps, down to
// one for a workgroup.  Parts of 8 steps at least, and the others empty, took longer: 2
// rows of 1000 in tables for 131072, 32 / 8 heads of 64, 8.4 us as it is and 10.6; 8 of
// 10 to 2000 in tables for 32768, 16 / 4 heads of 128, 9.0 and 12.3; one of 6000 in a
// table for 16384, 32 / 8 of 128, 11.7 and 14.6.
inline int64_t decode_splits(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t capacity)
{
    const int64_t rows = T * (Hq / Hk), units = B * Hk * ((rows + kDecodeRows - 1) / kDecodeRows);
    const int64_t steps = (capacity + kDecodeStep - 1) / kDecodeStep;
    int64_t n = (512 + units - 1) / units;
    if (n > (steps + 7) / 8) n = (steps + 7) / 8;
    return n < 1 ? 1 : n;
}
hipError_t launch_decode(const DecodeLaunch &a, hipStream_t stream);

}  // namespace attn
}  // namespace wkv7
