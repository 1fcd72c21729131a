// Host-side launchers of the int8 kernels and of the experts' operators, shared between the C-ABI layer
// and the kernel files.
#pragma once

#include "internal.h"

namespace w4a16 {

// Largest contraction of an int8 product: 128 * 128 * K stays below 2^31, so an int32 sum is exact.
constexpr int64_t kMaxW8K = 131056;
constexpr int kW8Chunk = 16;         // codes of one 16-byte load: rows are whole chunks
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;

// Rows of x (bf16, or fp32 when x_fp32) as int8 codes and one scale a row.
hipError_t launch_w8_quantize(const void* x, bool x_fp32, int8_t* codes, float* scales, int64_t R, int K,
                              hipStream_t stream);

enum class W8Epilogue {
    kStore,     // y = bf16(x_scale w_scale acc), or int32 partials
    kGlu,       // two weight sets: y = silu(g) * u
    kGluGrad    // two weight sets and dh: the gradients of both projections
};

// One product, or one per expert.  With offsets (int32 [E + 1], on the device) rows offsets[e] ..
// offsets[e + 1] - 1 take the e-th of E stacked weight matrices; row r's activations are row tokens[r]
// where tokens is given.
struct W8TileArgs {
    const uint16_t* x;         // decode kernel: bf16 activations [T, K], quantized on the way; else null
    const int8_t* a;           // codes of the activations [T, K]
    const float* a_scales;     // [T]
    const int8_t* w[2];        // weight sets [E, N, K]
    const float* w_scales[2];  // [E, N]
    const uint16_t* dh;        // kGluGrad [R, N]
    uint16_t* y[2];            // [R, N]; kGluGrad: the gradients of the gate and of the up projection
    uint16_t* scaled[2];       // kGluGrad: the same times the columns' scales, rows of ceil(N / 8) * 8
    int* ws;                   // int32 partials [split][M][N] when split > 1
    const int* offsets;
    const int* tokens;
    int E, T, R, N, K;
    int split;
    int height;                // rows of a tile, at most the shape's; 0: all of those
    int cut, cus;              // what is left of the tiles after whole rounds over `cus` compute units is cut into this
                               // many pieces of rows; experts: at most, as the kernel finds
};

// The transposed product: dx[r, k] = sum_s sum_n g_s[r, n] w_scale_s[n] w_s[n, k]; without w_scales the rows of
// g have the scales in them.
struct W8ColumnsArgs {
    const uint16_t* g[2];      // bf16 gradient rows, `pitch` values apart (a multiple of 8)
    const int8_t* w[2];        // weight sets [E, N, K]
    const float* w_scales[2];
    uint16_t* y;               // [R, K]
    float* ws;                 // fp32 partials [split][R][K] when split > 1
    const int* offsets;
    int E, R, N, K;
    int pitch, sets, split;
    int height, cut, cus;      // as above
};

struct W8TileShape {
    int bm, bn, waves;
    int grain;                 // rows of a tile count in steps of this
};
constexpr int kNumW8Tiles = 6, kNumW8PairTiles = 5;      // (the last one is not for two weight sets)
extern const W8TileShape kW8Tiles[kNumW8Tiles];
constexpr int kW8Step = 128;          // values of the contraction in one pipeline step
hipError_t launch_w8_tile(W8Epilogue epi, int tile, const W8TileArgs& args, hipStream_t stream);

// Decode rows (at most 16 of one matrix): workgroups of 16 weight rows whose `waves` waves take `share` lines of 128
// codes of the contraction each.
constexpr int kW8QmvRows = 16, kW8QmvColumns = 16, kW8QmvWaves = 16;
constexpr int kW8QuantizeRows = 2;      // rows that a workgroup quantizes for itself
struct W8QmvShape {
    int rows, waves, share;
    size_t lds;
};
// False where such workgroups are not possible (quantize: rows quantized by every workgroup for itself).
bool w8_qmv_shape(int rows, int waves, int K, bool quantize, W8QmvShape* out);
hipError_t launch_w8_qmv(const W8QmvShape& shape, const W8TileArgs& args, hipStream_t stream);

constexpr int kNumW8ColumnTiles = 3;
extern const W8TileShape kW8ColumnTiles[kNumW8ColumnTiles];
constexpr int kW8ColumnStep = 64;
hipError_t launch_w8_columns(int tile, const W8ColumnsArgs& args, hipStream_t stream);

// y = bf16(x_scale w_scale sum of the int32 partials [split][M][N]).
hipError_t launch_w8_sum(const int* ws, const float* a_scales, const float* w_scales, uint16_t* y, int64_t M, int N,
                         int split, hipStream_t stream);

// The router and the combination.
uint64_t experts_route_bytes(int64_t T, int E);
hipError_t launch_experts_route(const void* logits, bool fp32, int top_k, bool renormalize, float* weights, int* experts,
                                int* positions, int* tokens, int* offsets, int64_t T, int E, int* ws, hipStream_t stream);
hipError_t launch_experts_route_backward(const void* logits, bool fp32, const int* experts, const float* dweights,
                                         void* dlogits, int64_t T, int E, int top_k, bool renormalize,
                                         hipStream_t stream);
hipError_t launch_experts_combine(const uint16_t* y, const int* positions, const float* weights, uint16_t* out, int64_t T,
                                  int top_k, int64_t R, int N, hipStream_t stream);
hipError_t launch_experts_combine_backward(const uint16_t* dout, const uint16_t* y, const int* positions,
                                           const float* weights, uint16_t* dy, float* dweights, int64_t T, int top_k,
                                           int64_t R, int N, hipStream_t stream);

}  // namespace w4a16
