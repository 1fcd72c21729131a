// Launch policy of the int8 operators: which kernel, tile, height, split and pieces a call of given sizes takes.
// Pure host arithmetic.
#pragma once

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "abi_common.h"
#include "w8a8_internal.h"

namespace w4a16 {

constexpr int64_t kMaxRows = int64_t{1} << 30;      // rows and columns: tile and row numbers stay inside 31 bits
constexpr int64_t kMaxThreads = int64_t{1} << 32;   // threads of one launch stay below
constexpr int64_t kMaxTokens = int64_t{1} << 24;    // the router's and the combination's tokens

inline uint64_t round256(uint64_t v) { return (v + 255) / 256 * 256; }
inline int64_t padded(int64_t N) { return ceil_div(N, 8) * 8; }

inline bool is_backward(int32_t op) {
    return op == W8A8_LINEAR_BACKWARD || op == W8A8_EXPERTS_LINEAR_BACKWARD || op == W8A8_EXPERTS_GATE_UP_BACKWARD;
}
inline bool is_gated(int32_t op) { return op == W8A8_EXPERTS_GATE_UP || op == W8A8_EXPERTS_GATE_UP_BACKWARD; }
inline bool has_experts(int32_t op) { return op >= W8A8_EXPERTS_LINEAR; }

// Sizes of a call: E matrices [N, K], R rows of outputs, T rows of activations.
struct Sizes {
    int64_t E, T, R, N, K;
};

inline int check_matrix(int64_t R, int64_t K) {
    return R < 1 || R > kMaxRows || K < kW8Chunk || K > kMaxW8K || K % kW8Chunk != 0 ? W4A16_ERR_SHAPE : W4A16_OK;
}

inline int check_sizes(int32_t op, const Sizes& d, int32_t split_k) {
    if (op < W8A8_LINEAR || op > W8A8_EXPERTS_GATE_UP_BACKWARD) return W4A16_ERR_UNSUPPORTED;
    if (check_matrix(d.R, d.K) != W4A16_OK || check_matrix(d.T, d.K) != W4A16_OK) return W4A16_ERR_SHAPE;
    if (d.N < 1 || d.N > kMaxRows || d.E < 1 || d.E > kMaxExperts || split_k < 0) return W4A16_ERR_SHAPE;
    // the backward products contract over N
    if (is_backward(op) && d.N > kMaxK) return W4A16_ERR_SHAPE;
    if (has_experts(op)) return split_k > 1 ? W4A16_ERR_UNSUPPORTED : W4A16_OK;
    if (op == W8A8_LINEAR && d.T >= kMaxTokens) return W4A16_ERR_SHAPE;
    return d.E != 1 || d.T != d.R ? W4A16_ERR_SHAPE : W4A16_OK;
}

// Codes and scales of the activations, at the start of the workspace.
inline uint64_t activation_bytes(const Sizes& d) { return round256(static_cast<uint64_t>(d.T) * d.K) + round256(4 * static_cast<uint64_t>(d.T)); }
// Gradient rows in the workspace.  The transposed products read them sixteen bytes at a time: rows of another
// length are first copied, padded with zeros to eight values.  The gated pair's are made there, with the weights'
// scales in them.
inline uint64_t gradient_bytes(int32_t op, const Sizes& d) {
    if (!is_backward(op) || (!is_gated(op) && d.N % 8 == 0)) return 0;
    return (is_gated(op) ? 2 : 1) * round256(static_cast<uint64_t>(d.R) * padded(d.N) * 2);
}

struct Product {
    bool decode, quantize;   // the decode kernel; activations quantized in it
    W8QmvShape qmv;
    int tile, height, split, cut;
    int64_t M, N;            // output rows and columns
    int64_t blocks;          // workgroups of the launch, at most
    int cus;
};

// Microseconds of one tile: `fixed` for the first loads and the epilogue, and per pipeline step `base` and `grain` for
// every grain of its rows, alone on its compute unit; `beside` times that with a second one beside it (0: only one fits).
// Fitted to sweeps of every tile, height, split and cut on MI355X.  Behind the best form of another sweep, on average and at
// most: one matrix (22 shapes) 3.6 and 18% with weights from the caches, 3.3 and 19% from memory; transposed (12) 0.2 and 3%;
// experts (71 of shape and operator, from the caches) 3.3 and 30%.
struct TileCost {
    double fixed, base, grain, beside;
};
constexpr TileCost kTileCost[kNumW8Tiles] = {   // steps of 128 values
    // 128 x 128          256 x 256             64 x 128            128 x 256             64 x 256
    {5, 0.20, 0.13, 2.2}, {10, 0.42, 0.21, 0}, {4, 0.08, 0.17, 2}, {6, 0.36, 0.20, 0}, {5, 0.26, 0.20, 0},
    // 128 x 128, 8 waves
    {5, 0.22, 0.115, 0}};
constexpr TileCost kColumnCost[kNumW8ColumnTiles] = {   // steps of 64 values
    // 64 x 128         128 x 256             256 x 256
    {5, 0.25, 0.2, 2}, {6, 0.80, 0.02, 0}, {7, 0.75, 0.15, 0}};
// The gated pair's gradients: four outputs in place of one.
constexpr double kGradCost = 12;
// The transposed product of codes alone decodes faster.
constexpr double kUnscaled = 0.85;
// A split's second launch, and its partials per output.
constexpr double kSplitCost = 4.5, kPartialCost = 0.8e-6, kColumnPartialCost = 2.0e-6;
// Weights are as often in memory as in the caches that the sweeps found them in: per step, about half of what that costs.
constexpr double kColdStep = 0.08;
constexpr int64_t kMaxSplit = 8;
constexpr double kReadRate = 5.0e6;       // bytes of weights a microsecond

// Row tiles of a launch, as the launchers have it.
inline int64_t row_blocks(const Sizes& d, bool experts, int height) {
    return experts ? std::min(d.R, d.R / height + d.E) : ceil_div(d.R, height);
}

// Launches that share a tile's outputs among two kinds: whole rounds over the compute units, and the rest.
inline double rounds_time(double tiles, int64_t cus, const TileCost& c, double alone, double beside) {
    if (c.beside == 0) return std::ceil(tiles / static_cast<double>(cus)) * alone;
    const double slots = 2.0 * static_cast<double>(cus), whole = std::floor(tiles / slots), rest = tiles - whole * slots;
    return whole * beside + (rest == 0 ? 0 : rest <= static_cast<double>(cus) ? alone : beside);
}

// The decode kernel serves up to 16 rows of one matrix; above, and for experts, the tile, its height, the split and the
// pieces with the lowest modelled time.
inline Product product_of(int32_t op, const Sizes& d, int32_t split_k, int64_t cus, bool last) {
    Product p{};
    const bool experts = has_experts(op), back = is_backward(op) && last, grad = is_backward(op) && !last;
    p.M = d.R;
    p.N = back ? d.K : d.N;
    p.split = p.cut = 1;
    p.cus = static_cast<int>(cus);
    const int sets = is_gated(op) ? 2 : 1;
    if (!is_backward(op) && !experts && split_k == 0 && d.R <= kW8QmvRows) {
        // Waves: eight short shares where few workgroups have to bring everything on its way, fewer where there are many
        // (1 x 9728 x 2560: 8 waves 6.3 us, 4 6.3, 2 7.0; 100000 x 2560: 46, 47, 45; 2560 x 9728: 7.3, 9.7, 14.0).
        // Rows quantized on the way: one or two short ones (1 x 9728 x 2560 7.5 us, in two launches 9.3; 2 x 2560 x 9728
        // 10.1 and 10.4; 4 x 9728 x 2560 11.7 and 9.9).
        const int rows = static_cast<int>(d.R), K = static_cast<int>(d.K);
        const int64_t blocks = ceil_div(d.N, kW8QmvColumns);
        const int waves = blocks <= 2 * cus ? 8 : blocks <= 8 * cus ? 4 : 2;
        p.decode = true;
        p.quantize = op == W8A8_LINEAR && rows * d.K <= 16384 && w8_qmv_shape(rows, std::max(waves, (K + 2047) / 2048), K, true, &p.qmv);
        if (!p.quantize) w8_qmv_shape(rows, waves, K, false, &p.qmv);
        p.blocks = blocks;
        if (p.blocks * 64 * kW8QmvWaves < kMaxThreads) return p;
        p.decode = p.quantize = false;
    }
    const int64_t steps = back ? ceil_div(d.N, kW8ColumnStep) * sets : ceil_div(d.K, kW8Step);
    const int count = back ? kNumW8ColumnTiles : is_gated(op) ? kNumW8PairTiles : kNumW8Tiles;
    const double outputs = static_cast<double>(p.M) * p.N, pieces = static_cast<double>(std::min(d.E, d.R));
    const double memory = pieces * static_cast<double>(d.N) * d.K * sets / kReadRate;
    double best = 0;
    Product chosen = p;
    for (p.tile = 0; p.tile < count; ++p.tile) {
        const TileCost& c = back ? kColumnCost[p.tile] : kTileCost[p.tile];
        const W8TileShape& s = back ? kW8ColumnTiles[p.tile] : kW8Tiles[p.tile];
        const int64_t columns = ceil_div(p.N, !back && is_gated(op) ? s.bn / 2 : s.bn);
        const double fixed = c.fixed + (grad ? kGradCost : 0);
        auto step = [&](double rows) {
            return (c.base + c.grain * std::ceil(rows / s.grain)) * (back && sets > 1 ? kUnscaled : 1);
        };
        auto consider = [&](double t) {
            p.blocks = row_blocks(d, experts, p.height) * columns * p.split;
            if (experts || p.cut > 1) p.blocks += cus;
            if (best == 0 || t < best) {
                best = t;
                chosen = p;
            }
        };
        if (experts) {
            // an expert's rows: whole tiles, and one that ends somewhere
            p.height = s.bm;
            p.cut = std::max(1, back ? s.bm / 128 : s.bm / 64);
            const double mean = static_cast<double>(d.R) / pieces, n = static_cast<double>(steps);
            const double whole = std::max(0.0, mean / s.bm - 0.5);
            const double tile = (whole * (fixed + n * step(s.bm)) + fixed + n * step(std::min(mean, 0.5 * s.bm))) / (whole + 1);
            // (experts differ in how many rows they get, and one round lasts as long as its longest tile)
            const double longest = fixed + n * step(std::min(1.7 * mean, static_cast<double>(s.bm)));
            const double tiles = (whole > 0 ? 1.12 : 1) * pieces * static_cast<double>(columns) * (whole + 1), units = static_cast<double>(cus);
            const double rounds = tiles / (c.beside > 0 ? 2 * units : units), idle = std::ceil(rounds) - rounds;
            const double work = tile * (c.beside > 0 ? c.beside : 1) * (rounds + (c.beside > 0 ? 0.25 : p.cut > 1 && rounds > 2 ? 0.5 : 0.75) * idle);
            // (two workgroups a compute unit wait for the weights less; of two forms that wait the one with less work)
            consider(std::max({tiles <= units ? longest : work, longest, memory * (c.beside > 0 ? 1 : 1.12)}) + 1e-3 * work);
            continue;
        }
        for (p.height = s.bm; p.height > s.bm - 3 * s.grain && p.height > 0; p.height -= s.grain) {
            const double tiles = static_cast<double>(ceil_div(d.R, p.height) * columns);
            const double rows = static_cast<double>(std::min<int64_t>(p.height, d.R));
            const int64_t most = last ? std::min(kMaxSplit, steps) : 1;
            const int64_t first = split_k > 0 && most > 1 ? std::min<int64_t>(split_k, steps) : 1;
            for (int64_t z = first; z <= (split_k > 0 ? first : most); ++z) {
                const double n = static_cast<double>(ceil_div(steps, z));
                const double alone = fixed + n * step(rows), beside = fixed + n * step(rows) * c.beside;
                double t = rounds_time(tiles * static_cast<double>(z), cus, c, alone, beside);
                if (z > 1) t += kSplitCost + (back ? kColumnPartialCost : kPartialCost) * outputs * static_cast<double>(z);
                t += kColdStep * n;
                p.split = static_cast<int>(z);
                p.cut = 1;
                consider(std::max(t, memory));
                // the last round's tiles in two or four pieces of rows
                const double round = static_cast<double>(c.beside > 0 ? 2 * cus : cus);
                const double rest = tiles - std::floor(tiles / static_cast<double>(cus)) * static_cast<double>(cus);
                for (p.cut = 2; z == 1 && p.cut <= 4 && tiles > static_cast<double>(cus); p.cut *= 2) {
                    if (rest == 0 || rest * p.cut > round || p.height / p.cut < s.grain) continue;
                    const double low = fixed + n * step(std::ceil(rows / p.cut)) * (rest * p.cut > static_cast<double>(cus) ? c.beside : 1);
                    consider(std::max(rounds_time(tiles - rest, cus, c, alone, beside) + low + kColdStep * n, memory));
                }
            }
            p.split = p.cut = 1;
        }
    }
    return chosen;
}

// The gated backward's first launch: both projections once more, with another tile and grid than dx has.
inline Product both_again(const Sizes& d, int64_t cus) { return product_of(W8A8_EXPERTS_GATE_UP_BACKWARD, d, 0, cus, false); }

}  // namespace w4a16
