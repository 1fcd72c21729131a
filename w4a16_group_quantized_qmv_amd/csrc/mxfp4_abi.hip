// MXFP4 entry points of include/w4a16.h: argument checks, the launch policy and the calls.  As in
// abi.hip every compute call only enqueues kernels on the caller's stream, allocates nothing and
// reports by status.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "abi_common.h"
#include "mxfp4_internal.h"

namespace {

using namespace w4a16;

// Rows and columns: a tile's row and column numbers stay inside 31 bits.
constexpr int64_t kMaxMxDim = int64_t{1} << 30;
constexpr int64_t kMaxThreads = int64_t{1} << 32;   // threads of one launch stay below

uint64_t round256(uint64_t v) { return (v + 255) / 256 * 256; }

int check_rows(int64_t R, int64_t K) {
    if (R < 1 || R > kMaxMxDim || K < 1 || K > kMaxK || K % kMxBlock != 0) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

bool is_backward(int32_t op) { return op == MXFP4_LINEAR_BACKWARD || op == MXFP4_GATE_UP_BACKWARD; }

int check_op(int32_t op, int64_t M, int64_t N, int64_t K, int32_t split_k) {
    if (op < MXFP4_LINEAR || op > MXFP4_GATE_UP_BACKWARD) return W4A16_ERR_UNSUPPORTED;
    if (check_rows(M, K) != W4A16_OK || N < 1 || N > kMaxMxDim || split_k < 0) return W4A16_ERR_SHAPE;
    // the backward products contract over N: their gradient rows obey the limit of the contraction
    if (is_backward(op) && N > kMaxK) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

uint64_t code_bytes(int64_t R, int64_t K) { return static_cast<uint64_t>(R) * (K / 2); }
uint64_t scale_bytes(int64_t R, int64_t K) { return static_cast<uint64_t>(R) * (K / kMxBlock); }
// Activation codes and scales of mxfp4a4_linear, at the start of its workspace.
uint64_t activation_bytes(int64_t M, int64_t K) { return round256(code_bytes(M, K)) + round256(scale_bytes(M, K)); }

// The backward products read gradient rows sixteen bytes at a time: rows of another length are first
// copied to the start of the workspace, padded with zeros to eight values.
int64_t padded(int64_t N) { return ceil_div(N, 8) * 8; }
uint64_t padding_bytes(int32_t op, int64_t M, int64_t N) {
    if (!is_backward(op) || N % 8 == 0) return 0;
    return (op == MXFP4_GATE_UP_BACKWARD ? 2 : 1) * round256(static_cast<uint64_t>(M) * padded(N) * 2);
}
// The decode kernel serves the forward operators at up to 16 rows, unless a split is asked for (or
// four columns per workgroup would make too large a launch); it needs no workspace (4-bit activations
// are quantized on the way).
bool decodes(int32_t op, int64_t M, int64_t N, int32_t split_k) {
    return M <= kMxQmvRows && !is_backward(op) && split_k == 0 && ceil_div(N, 4) * 64 * kMxQmvWaves < kMaxThreads;
}
// Workspace that an operator cannot do without (the rest is for partials).
uint64_t fixed_bytes(int32_t op, int64_t M, int64_t N, int64_t K, int32_t split_k) {
    if (op == MXFP4A4_LINEAR) return decodes(op, M, N, split_k) ? 0 : activation_bytes(M, K);
    return padding_bytes(op, M, N);
}

struct Product {
    MxOperands operands;
    MxEpilogue epilogue;
    int64_t M, N, L;     // output rows and columns, contraction length
    int sets;            // weight sets
    int tile;
    int split;
    bool decode;         // the decode kernel
    int cus;
};

// The product that an operator's last launch computes.
Product product_of(int32_t op, int64_t M, int64_t N, int64_t K) {
    switch (op) {
        case MXFP4_LINEAR: return {MxOperands::kRows, MxEpilogue::kStore, M, N, K, 1, 0, 1, false, 0};
        case MXFP4_LINEAR_BACKWARD: return {MxOperands::kColumns, MxEpilogue::kStore, M, K, N, 1, 0, 1, false, 0};
        case MXFP4_GATE_UP: return {MxOperands::kRows, MxEpilogue::kGlu, M, N, K, 2, 0, 1, false, 0};
        case MXFP4_GATE_UP_BACKWARD: return {MxOperands::kColumns, MxEpilogue::kStore, M, K, N, 2, 0, 1, false, 0};
        default: return {MxOperands::kCodes, MxEpilogue::kStore, M, N, K, 1, 0, 1, false, 0};
    }
}

int64_t tiles_of(const Product& p) {
    const MxTileShape& s = kMxTiles[p.tile];
    return ceil_div(p.M, s.bm) * ceil_div(p.N, p.epilogue == MxEpilogue::kStore ? s.bn : s.bn / 2);
}

// Pipeline units of the contraction: what split-K distributes.
int64_t units_of(const Product& p) {
    return ceil_div(p.L, mx_unit(p.operands)) * (p.operands == MxOperands::kColumns ? p.sets : 1);
}

// Microseconds of one tile on a compute unit, fitted to sweeps of every tile and split on MI355X (24 to
// 4096 rows; 2560 x 9728, 9728 x 2560, 4096 x 2560 and 1024 x 2560 weights): `fixed` for the first
// loads and the epilogue, and `step` per pipeline step, alone on its compute unit and (for the tiles
// of which two fit) with a second one beside it.  64 x 128 tiles of codes take 106496 of the 163840 bytes
// of LDS, so a second one waits (58 x 42636 x 1216 with codes: 334 of them 21.3 us, two rounds; 128 x 128
// 15.9).
struct TileCost {
    double fixed, step, step_beside;
};
constexpr TileCost kTileCost[3][kNumMxTiles] = {
    // 128 x 128        256 x 256      64 x 128          192 x 256       128 x 256
    {{3.0, 0.67, 1.2}, {9.0, 1.20, 0}, {4.5, 0.41, 0}, {6.0, 1.05, 0}, {5.0, 1.05, 0}},       // kCodes (256 values a step)
    {{5.0, 0.46, 1.0}, {10.0, 1.30, 0}, {5.0, 0.32, 0.54}, {8.0, 1.17, 0}, {6.0, 0.80, 0}},   // kRows (64)
    {{5.0, 0.64, 0.9}, {8.0, 1.42, 0}, {5.0, 0.54, 0.9}, {6.0, 1.32, 0}, {5.0, 0.88, 0}},     // kColumns (64)
};
// A split's second launch, and its partials written and read per output (8 bytes at about 4 TB/s).
constexpr double kSplitCost = 3.5, kPartialCost = 2e-6;
constexpr int64_t kMaxSplit = 8;

// The tile and the split with the lowest modelled time.  Against the best of a sweep of every tile and
// split on 63 shapes the choice is behind by, on average and at worst, 0.4% and 3% with kRows, 1.0% and 11%
// with kColumns (1500 rows of 6000 x 2048: 56 us in two slices of 128 x 256, 51 in four of 192 x 256) and
// 2.2% and 12% with kCodes (24 rows of 151936 x 2560: 44 us in 64 x 128 tiles, 39 in 128 x 128).
void choose(Product& p, int32_t split_k, int64_t cus) {
    if (p.decode) return;
    const int64_t units = units_of(p);
    const int64_t steps = ceil_div(p.L, mx_step(p.operands)) * (p.operands == MxOperands::kColumns ? p.sets : 1);
    const double outputs = static_cast<double>(p.M) * p.N * (p.epilogue == MxEpilogue::kGlu ? 2 : 1);
    double best = 0;
    Product chosen = p;
    for (p.tile = 0; p.tile < kNumMxTiles; ++p.tile) {
        const TileCost& c = kTileCost[static_cast<int>(p.operands)][p.tile];
        const int64_t tiles = tiles_of(p);
        const int64_t first = split_k > 0 ? std::min<int64_t>(split_k, units) : 1;
        const int64_t last = split_k > 0 ? first : std::min(kMaxSplit, units);
        for (int64_t s = first; s <= last; ++s) {
            const bool beside = c.step_beside > 0 && tiles * s > cus;
            const double rounds = static_cast<double>(ceil_div(tiles * s, beside ? 2 * cus : cus));
            double t = rounds * (c.fixed + static_cast<double>(ceil_div(steps, s)) * (beside ? c.step_beside : c.step));
            if (s > 1) t += kSplitCost + kPartialCost * outputs * static_cast<double>(s);
            if (best == 0 || t < best) {
                best = t;
                chosen = p;
                chosen.split = static_cast<int>(s);
            }
        }
    }
    p = chosen;
}

uint64_t partial_bytes(const Product& p) {
    if (p.split == 1) return 0;
    return static_cast<uint64_t>(p.epilogue == MxEpilogue::kGlu ? 2 : 1) * p.split * p.M * p.N * sizeof(float);
}

int make_plan(int32_t op, int64_t M, int64_t N, int64_t K, int32_t split_k, int32_t num_cus, w4a16_plan_t* out,
              Product* product = nullptr) {
    if (!out) return W4A16_ERR_NULL;
    int st = check_op(op, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    int32_t cus = num_cus;
    if (cus <= 0) {
        st = query_num_cus(&cus);
        if (st != W4A16_OK) return st;
    }
    Product p = product_of(op, M, N, K);
    p.decode = decodes(op, M, N, split_k);
    p.cus = cus;
    choose(p, split_k, cus);
    const MxTileShape& s = kMxTiles[p.tile];
    if (!p.decode && (tiles_of(p) * p.split * 64 * s.waves >= kMaxThreads ||
                      (p.split > 1 && ceil_div(p.M * p.N, 4) >= kMaxThreads)))
        return W4A16_ERR_SHAPE;
    out->path = W4A16_PATH_MXFP4;
    out->tile_m = s.bm;
    out->tile_n = p.epilogue == MxEpilogue::kStore ? s.bn : s.bn / 2;
    out->tile_k = mx_step(p.operands);
    out->grid_x = static_cast<int32_t>(ceil_div(p.N, out->tile_n));
    out->grid_y = static_cast<int32_t>(ceil_div(p.M, s.bm));
    out->grid_z = p.split;
    out->block_threads = 64 * s.waves;
    out->split_k = p.split;
    out->k_waves = 1;
    out->num_cus = cus;
    out->variant = p.tile;
    if (p.decode) {
        MxQmvShape q;
        mx_qmv_shape(p.operands, p.sets, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), cus, true, &q);
        out->path = W4A16_PATH_MXFP4_QMV;
        out->tile_m = q.rows;
        out->tile_n = q.columns;
        out->tile_k = kMxBlock;
        out->grid_x = q.groups;
        out->grid_y = 1;
        out->block_threads = 64 * q.waves;
        out->k_waves = q.wide ? 1 : q.waves;
        out->variant = q.wide ? 0 : q.batch;
    }
    out->workspace_bytes = fixed_bytes(op, M, N, K, split_k) + partial_bytes(p);
    if (product) *product = p;
    return W4A16_OK;
}

// A weight set (or an operand in codes) of R rows: non-null codes on 16 bytes.
int check_codes(const uint8_t* codes, const uint8_t* scales) {
    if (!codes || !scales) return W4A16_ERR_NULL;
    return aligned(codes, 16) ? W4A16_OK : W4A16_ERR_ALIGN;
}

bool overlaps_codes(const void* y, uint64_t ny, const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t K) {
    return overlaps(y, ny, codes, code_bytes(R, K)) || overlaps(y, ny, scales, scale_bytes(R, K));
}

// The plan fitted to the workspace, before any launch: without room a policy split is dropped and a
// forced one is an error; the operator's fixed part has to fit.
int fit(int32_t op, int64_t M, int64_t N, int64_t K, int32_t split_k, const void* workspace, size_t workspace_bytes,
        Product* p) {
    const uint64_t used = fixed_bytes(op, M, N, K, split_k);
    const bool usable = workspace && aligned(workspace, 16);
    const int missing = workspace && !usable ? W4A16_ERR_ALIGN : W4A16_ERR_WORKSPACE;
    if (used > 0 && (!usable || workspace_bytes < used)) return missing;
    w4a16_plan_t plan;
    const int st = make_plan(op, M, N, K, split_k, 0, &plan, p);
    if (st != W4A16_OK) return st;
    if (p->split > 1 && (!usable || workspace_bytes - used < partial_bytes(*p))) {
        if (split_k > 1) return missing;
        return make_plan(op, M, N, K, 1, 0, &plan, p);
    }
    return W4A16_OK;
}

// Launch a fitted product and sum its slices; partials: the workspace after the fixed part.
int run_product(const Product& p, MxTileArgs args, void* partials, hipStream_t stream, bool quantize = false) {
    args.M = static_cast<int>(p.M);
    args.N = static_cast<int>(p.N);
    args.L = static_cast<int>(p.L);
    args.sets = p.sets;
    args.split = p.split;
    args.ws = static_cast<float*>(partials);
    if (args.pitch == 0) args.pitch = p.operands == MxOperands::kCodes ? p.L / 2 : 2 * p.L;
    if (p.decode) return to_status(launch_mx_qmv(p.operands, p.epilogue, quantize, args, p.cus, stream));
    hipError_t e = launch_mx_tile(p.operands, p.epilogue, p.tile, args, stream);
    if (e != hipSuccess || p.split == 1) return to_status(e);
    return to_status(launch_mx_sum(args.ws, args.y[0], p.epilogue == MxEpilogue::kGlu ? 2 : 1, p.M * p.N, p.split, stream));
}

void* after(void* workspace, uint64_t bytes) {
    return workspace ? static_cast<uint8_t*>(workspace) + bytes : nullptr;
}

// Gradient rows [M, N] as 16-byte rows: themselves, or their padded copy at `copy`.
int pad_gradient(const uint16_t* dy, int64_t M, int64_t N, void* copy, hipStream_t stream, const void** rows) {
    *rows = dy;
    if (N % 8 == 0) return W4A16_OK;
    *rows = copy;
    return to_status(launch_mx_pad_rows(dy, static_cast<uint16_t*>(copy), M, static_cast<int>(N), stream));
}

int run_linear(int32_t op, const uint16_t* x, const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t M,
               int64_t N, int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_op(op, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    if (!x || !y) return W4A16_ERR_NULL;
    st = check_codes(codes, scales);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(y, 2)) return W4A16_ERR_ALIGN;
    const bool back = is_backward(op);
    const uint64_t ny = static_cast<uint64_t>(M) * (back ? K : N) * 2, nx = static_cast<uint64_t>(M) * (back ? N : K) * 2;
    if (overlaps(y, ny, x, nx) || overlaps_codes(y, ny, codes, scales, N, K)) return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(op, M, N, K, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MxTileArgs args{};
    args.a[0] = x;
    if (back) {
        st = pad_gradient(x, M, N, workspace, s, &args.a[0]);
        if (st != W4A16_OK) return st;
        args.pitch = 2 * padded(N);
    }
    args.w[0] = codes;
    args.w_scales[0] = scales;
    args.y[0] = y;
    return run_product(p, args, after(workspace, fixed_bytes(op, M, N, K, split_k)), s);
}

}  // namespace

extern "C" {

int mxfp4_quantize_rows(const void* x, int32_t x_type, uint8_t* codes, uint8_t* scales, int64_t R, int64_t K,
                        void* stream) {
    const int st = check_rows(R, K);
    if (st != W4A16_OK) return st;
    if (x_type != MXFP4_BF16 && x_type != MXFP4_FP32) return W4A16_ERR_UNSUPPORTED;
    if (!x || !codes || !scales) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(codes, 16)) return W4A16_ERR_ALIGN;
    const uint64_t nx = static_cast<uint64_t>(R) * K * (x_type == MXFP4_FP32 ? 4 : 2);
    if (overlaps_codes(x, nx, codes, scales, R, K) ||
        overlaps(codes, code_bytes(R, K), scales, scale_bytes(R, K)))
        return W4A16_ERR_OVERLAP;
    return to_status(launch_mx_quantize(x, x_type == MXFP4_FP32, codes, scales, R * (K / kMxBlock),
                                        static_cast<hipStream_t>(stream)));
}

int mxfp4_dequantize_rows(const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t R, int64_t K,
                          void* stream) {
    int st = check_rows(R, K);
    if (st != W4A16_OK) return st;
    if (!y) return W4A16_ERR_NULL;
    st = check_codes(codes, scales);
    if (st != W4A16_OK) return st;
    if (!aligned(y, 16)) return W4A16_ERR_ALIGN;
    if (overlaps_codes(y, static_cast<uint64_t>(R) * K * 2, codes, scales, R, K)) return W4A16_ERR_OVERLAP;
    return to_status(launch_mx_dequantize(codes, scales, y, R * (K / kMxBlock), static_cast<hipStream_t>(stream)));
}

int mxfp4_plan(int32_t op, int64_t M, int64_t N, int64_t K, int32_t split_k, int32_t num_cus, w4a16_plan_t* out) {
    return make_plan(op, M, N, K, split_k, num_cus, out);
}

int mxfp4_linear(const uint16_t* x, const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t M, int64_t N,
                 int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    return run_linear(MXFP4_LINEAR, x, codes, scales, y, M, N, K, split_k, workspace, workspace_bytes, stream);
}

int mxfp4_linear_backward(const uint16_t* dy, const uint8_t* codes, const uint8_t* scales, uint16_t* dx, int64_t M,
                          int64_t N, int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes,
                          void* stream) {
    return run_linear(MXFP4_LINEAR_BACKWARD, dy, codes, scales, dx, M, N, K, split_k, workspace, workspace_bytes, stream);
}

int qmm_mxfp4a4(const uint8_t* xq, const uint8_t* xs, const uint8_t* codes, const uint8_t* scales, uint16_t* y,
                int64_t M, int64_t N, int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes,
                void* stream) {
    int st = check_op(MXFP4_QMM_A4, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    st = check_codes(xq, xs);
    if (st == W4A16_OK) st = check_codes(codes, scales);
    if (st != W4A16_OK) return st;
    if (!y) return W4A16_ERR_NULL;
    if (!aligned(y, 2)) return W4A16_ERR_ALIGN;
    const uint64_t ny = static_cast<uint64_t>(M) * N * 2;
    if (overlaps_codes(y, ny, xq, xs, M, K) || overlaps_codes(y, ny, codes, scales, N, K)) return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(MXFP4_QMM_A4, M, N, K, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    MxTileArgs args{};
    args.a[0] = xq;
    args.a_scales = xs;
    args.w[0] = codes;
    args.w_scales[0] = scales;
    args.y[0] = y;
    return run_product(p, args, workspace, static_cast<hipStream_t>(stream));
}

int mxfp4a4_linear(const uint16_t* x, const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t M, int64_t N,
                   int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_op(MXFP4A4_LINEAR, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    if (!x || !y) return W4A16_ERR_NULL;
    st = check_codes(codes, scales);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(y, 2)) return W4A16_ERR_ALIGN;
    const uint64_t ny = static_cast<uint64_t>(M) * N * 2;
    if (overlaps(y, ny, x, static_cast<uint64_t>(M) * K * 2) || overlaps_codes(y, ny, codes, scales, N, K))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(MXFP4A4_LINEAR, M, N, K, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MxTileArgs args{};
    args.w[0] = codes;
    args.w_scales[0] = scales;
    args.y[0] = y;
    if (p.decode) {
        args.a[0] = x;
        args.pitch = 2 * K;
        return run_product(p, args, nullptr, s, true);
    }
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + round256(code_bytes(M, K));
    const hipError_t e = launch_mx_quantize(x, false, xq, xs, M * (K / kMxBlock), s);
    if (e != hipSuccess) return to_status(e);
    args.a[0] = xq;
    args.a_scales = xs;
    return run_product(p, args, after(workspace, activation_bytes(M, K)), s);
}

int mxfp4_gate_up_swiglu(const uint16_t* x, const uint8_t* codes_gate, const uint8_t* scales_gate,
                         const uint8_t* codes_up, const uint8_t* scales_up, uint16_t* h, int64_t M, int64_t N,
                         int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_op(MXFP4_GATE_UP, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    if (!x || !h) return W4A16_ERR_NULL;
    st = check_codes(codes_gate, scales_gate);
    if (st == W4A16_OK) st = check_codes(codes_up, scales_up);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(h, 2)) return W4A16_ERR_ALIGN;
    const uint64_t nh = static_cast<uint64_t>(M) * N * 2;
    if (overlaps(h, nh, x, static_cast<uint64_t>(M) * K * 2) || overlaps_codes(h, nh, codes_gate, scales_gate, N, K) ||
        overlaps_codes(h, nh, codes_up, scales_up, N, K))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(MXFP4_GATE_UP, M, N, K, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    MxTileArgs args{};
    args.a[0] = x;
    args.w[0] = codes_gate;
    args.w[1] = codes_up;
    args.w_scales[0] = scales_gate;
    args.w_scales[1] = scales_up;
    args.y[0] = h;
    return run_product(p, args, workspace, static_cast<hipStream_t>(stream));
}

int mxfp4_gate_up_swiglu_backward(const uint16_t* x, const uint8_t* codes_gate, const uint8_t* scales_gate,
                                  const uint8_t* codes_up, const uint8_t* scales_up, const uint16_t* dh, uint16_t* dx,
                                  uint16_t* dgate, uint16_t* dup, int64_t M, int64_t N, int64_t K, int32_t split_k,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_op(MXFP4_GATE_UP_BACKWARD, M, N, K, split_k);
    if (st != W4A16_OK) return st;
    if (!x || !dh || !dx || !dgate || !dup) return W4A16_ERR_NULL;
    st = check_codes(codes_gate, scales_gate);
    if (st == W4A16_OK) st = check_codes(codes_up, scales_up);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(dgate, 16) || !aligned(dup, 16) || !aligned(dh, 2) || !aligned(dx, 2))
        return W4A16_ERR_ALIGN;
    const uint64_t mk = static_cast<uint64_t>(M) * K * 2, mn = static_cast<uint64_t>(M) * N * 2;
    const struct {
        const void* p;
        uint64_t n;
    } out[3] = {{dx, mk}, {dgate, mn}, {dup, mn}};
    for (int i = 0; i < 3; ++i) {
        if (overlaps(out[i].p, out[i].n, x, mk) || overlaps(out[i].p, out[i].n, dh, mn) ||
            overlaps_codes(out[i].p, out[i].n, codes_gate, scales_gate, N, K) ||
            overlaps_codes(out[i].p, out[i].n, codes_up, scales_up, N, K))
            return W4A16_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return W4A16_ERR_OVERLAP;
    }
    // both launches' plans before the first: every refusal comes before any work
    Product dx_product, again;
    st = fit(MXFP4_GATE_UP_BACKWARD, M, N, K, split_k, workspace, workspace_bytes, &dx_product);
    if (st == W4A16_OK) st = fit(MXFP4_GATE_UP, M, N, K, 1, nullptr, 0, &again);
    if (st != W4A16_OK) return st;
    again.epilogue = MxEpilogue::kGluGrad;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MxTileArgs args{};
    args.a[0] = x;
    args.w[0] = codes_gate;
    args.w[1] = codes_up;
    args.w_scales[0] = scales_gate;
    args.w_scales[1] = scales_up;
    args.dh = dh;
    args.y[0] = dgate;
    args.y[1] = dup;
    st = run_product(again, args, nullptr, s);
    if (st != W4A16_OK) return st;
    // dx from dgate and dup as the caller gets them, rounded to bf16: the matrix cores take 16 bits, and so
    // dx is the input gradient of the two projections for exactly those gradients (as two
    // mxfp4_linear_backward calls would have it).  Each factor is off by up to 2^-8
    // of itself, which takes dx's error against 64 bits from 0.0017 (its own rounding; relative,
    // root mean square) to 0.0023.  Keeping the remainders as second bf16 operands would double the
    // product, 364 of 742 us at 4096 x 9728 x 2560, and need twice the gradients' memory.
    const uint64_t pad = padding_bytes(MXFP4_GATE_UP_BACKWARD, M, N);
    st = pad_gradient(dgate, M, N, workspace, s, &args.a[0]);
    if (st == W4A16_OK) st = pad_gradient(dup, M, N, after(workspace, pad / 2), s, &args.a[1]);
    if (st != W4A16_OK) return st;
    args.pitch = 2 * padded(N);
    args.y[0] = dx;
    return run_product(dx_product, args, after(workspace, pad), s);
}

}  // extern "C"
