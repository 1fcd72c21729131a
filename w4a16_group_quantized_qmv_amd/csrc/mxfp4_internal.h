// Host-side launchers of the MXFP4 kernels, shared between the C-ABI layer and the kernel files.
#pragma once

#include "internal.h"

namespace w4a16 {

constexpr int kMxBlock = 32;   // values of one block

// Rows of x (bf16, or fp32 when x_fp32) as `blocks` consecutive blocks of 32 values.
hipError_t launch_mx_quantize(const void* x, bool x_fp32, uint8_t* codes, uint8_t* scales, int64_t blocks,
                              hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t blocks,
                                hipStream_t stream);

// Rows of N bf16 values as rows of ceil(N / 8) * 8, the rest zeros.
hipError_t launch_mx_pad_rows(const uint16_t* x, uint16_t* y, int64_t M, int N, hipStream_t stream);

// Sums of split-K partials [sets][split][MN], in slice order: y = bf16(sum), or silu(sum) * sum of two.
hipError_t launch_mx_sum(const float* ws, uint16_t* y, int sets, int64_t MN, int split, hipStream_t stream);

// What a tile multiplies.
enum class MxOperands {
    kCodes,     // MXFP4 rows by MXFP4 rows, on the scaled matrix cores
    kRows,      // bf16 rows by MXFP4 rows, contracted along the blocks
    kColumns    // bf16 rows by MXFP4 columns: contracted across the weight rows
};
// What a tile does with the products.
enum class MxEpilogue {
    kStore,     // y = bf16(acc), or fp32 partials
    kGlu,       // two weight sets: y = silu(g) * u
    kGluGrad    // two weight sets and dh: the gradients of both projections
};

struct MxTileArgs {
    const void* a[2];          // rows of the left operand (kColumns: one per weight set)
    int64_t pitch;             // bytes of one of its rows
    const uint8_t* a_scales;   // kCodes
    const uint8_t* w[2];       // codes of the weight sets
    const uint8_t* w_scales[2];
    const uint16_t* dh;        // kGluGrad
    uint16_t* y[2];            // output; kGluGrad: the gradients of the gate and of the up projection
    float* ws;                 // fp32 partials [weight set][split][M][N] when split > 1
    int M, N, L;               // output rows, output columns (of one weight set), contraction length
    int sets;                  // weight sets (kColumns: summed over)
    int split;                 // slices of the contraction
};

struct MxTileShape {
    int bm, bn, waves;         // rows and weight rows of a workgroup's tile
};
constexpr int kNumMxTiles = 5;
extern const MxTileShape kMxTiles[kNumMxTiles];
// Values of the contraction in one pipeline step, and in the unit that split-K distributes (a pair of
// steps where two steps' weights or scales are loaded together).
inline int mx_step(MxOperands op) { return op == MxOperands::kCodes ? 256 : 64; }
inline int mx_unit(MxOperands op) { return op == MxOperands::kCodes ? 512 : op == MxOperands::kRows ? 128 : 64; }

// Decode rows (at most 16).  `groups` workgroups.  Wide form: eight waves of 16-column blocks.  Else
// workgroups of `columns` weight rows whose `waves` waves take `share` units (1 KB of codes) of the
// contraction each, `batch` of them in flight; `rows` activation row slots.  `lds` dynamic bytes.
// whole: the scale rows start on 16 bytes (the wide form loads them so).
constexpr int kMxQmvRows = 16;
constexpr int kMxQmvWaves = 16;
constexpr int kMxWideWaves = 8;
struct MxQmvShape {
    bool wide;
    int groups, rows, columns, waves, share, batch;
    size_t lds;
};
bool mx_qmv_shape(MxOperands op, int sets, int M, int N, int K, int cus, bool whole, MxQmvShape* out);
// quantize (kCodes): the activations are bf16 rows, quantized on the way.
hipError_t launch_mx_qmv(MxOperands op, MxEpilogue epi, bool quantize, const MxTileArgs& args, int cus,
                         hipStream_t stream);

hipError_t launch_mx_tile(MxOperands op, MxEpilogue epi, int tile, const MxTileArgs& args, hipStream_t stream);

}  // namespace w4a16
