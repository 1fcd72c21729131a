// Entry points of include/w4a16.h for int8 weights and for mixtures of experts: argument checks, the launch
// policy and the calls.  As in abi.hip every compute call only enqueues kernels on the caller's stream,
// allocates nothing and reports by status.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <stdint.h>

#include "abi_common.h"
#include "mxfp4_internal.h"
#include "w8a8_policy.h"

namespace {

using namespace w4a16;

uint64_t partial_bytes(const Product& p) { return p.split == 1 ? 0 : static_cast<uint64_t>(p.split) * p.M * p.N * 4; }

// Workspace that an operator cannot do without (the rest is for partials).
uint64_t fixed_bytes(int32_t op, const Sizes& d, const Product& p) {
    const bool quantizes = op == W8A8_LINEAR || op == W8A8_EXPERTS_LINEAR || is_gated(op);
    return (quantizes && !p.quantize ? activation_bytes(d) : 0) + gradient_bytes(op, d);
}

int plan_call(int32_t op, const Sizes& d, int32_t split_k, int32_t num_cus, Product* p, int32_t* used_cus) {
    int st = check_sizes(op, d, split_k);
    if (st != W4A16_OK) return st;
    int32_t cus = num_cus;
    if (cus <= 0) {
        st = query_num_cus(&cus);
        if (st != W4A16_OK) return st;
    }
    *used_cus = cus;
    *p = product_of(op, d, split_k, cus, true);
    const W8TileShape& s = is_backward(op) ? kW8ColumnTiles[p->tile] : kW8Tiles[p->tile];
    if (!p->decode && (p->blocks * 64 * s.waves >= kMaxThreads ||
                       (p->split > 1 && ceil_div(p->M * p->N, 4) >= kMaxThreads)))
        return W4A16_ERR_SHAPE;
    if (op == W8A8_EXPERTS_GATE_UP_BACKWARD) {
        const Product again = both_again(d, cus);
        if (again.blocks * 64 * kW8Tiles[again.tile].waves >= kMaxThreads) return W4A16_ERR_SHAPE;
    }
    return W4A16_OK;
}

struct Range {
    const void* p;
    uint64_t n;
};

// No output shares bytes with an input or with another output.
bool disjoint(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
    for (const Range* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Range& i : inputs)
            if (i.p && overlaps(o->p, o->n, i.p, i.n)) return false;
        for (const Range* q = outputs.begin(); q != o; ++q)
            if (overlaps(o->p, o->n, q->p, q->n)) return false;
    }
    return true;
}

int check_weights(const int8_t* codes, const float* scales) {
    if (!codes || !scales) return W4A16_ERR_NULL;
    return aligned(codes, 16) && aligned(scales, 4) ? W4A16_OK : W4A16_ERR_ALIGN;
}

// The plan fitted to the workspace, before any launch: without room a policy split is dropped and a forced one
// is an error; the operator's fixed part has to fit.
int fit(int32_t op, const Sizes& d, int32_t split_k, const void* workspace, size_t workspace_bytes, Product* p) {
    int32_t cus;
    const int st = plan_call(op, d, split_k, 0, p, &cus);
    if (st != W4A16_OK) return st;
    const uint64_t used = fixed_bytes(op, d, *p);
    const bool usable = workspace && aligned(workspace, 16);
    const int missing = workspace && !usable ? W4A16_ERR_ALIGN : W4A16_ERR_WORKSPACE;
    if (used > 0 && (!usable || workspace_bytes < used)) return missing;
    if (p->split > 1 && (!usable || workspace_bytes - used < partial_bytes(*p))) {
        if (split_k > 1) return missing;
        return plan_call(op, d, 1, 0, p, &cus);
    }
    return W4A16_OK;
}

void* after(void* workspace, uint64_t bytes) {
    return workspace ? static_cast<uint8_t*>(workspace) + bytes : nullptr;
}

W8TileArgs tile_args(const Sizes& d, const Product& p, const int32_t* offsets, const int32_t* tokens, uint16_t* y) {
    W8TileArgs a{};
    a.offsets = offsets;
    a.tokens = tokens;
    a.E = static_cast<int>(d.E);
    a.T = static_cast<int>(d.T);
    a.R = static_cast<int>(d.R);
    a.N = static_cast<int>(d.N);
    a.K = static_cast<int>(d.K);
    a.split = p.split;
    a.height = p.height;
    a.cut = p.cut;
    a.cus = p.cus;
    a.y[0] = y;
    return a;
}

// A forward product of codes (or, where the plan says so, of bf16 rows): the kernel and a split's sum.
int run_forward(W8Epilogue epi, const Product& p, W8TileArgs& args, void* partials, hipStream_t stream) {
    args.ws = static_cast<int*>(partials);
    if (p.decode) return to_status(launch_w8_qmv(p.qmv, args, stream));
    const hipError_t e = launch_w8_tile(epi, p.tile, args, stream);
    if (e != hipSuccess || p.split == 1) return to_status(e);
    return to_status(launch_w8_sum(args.ws, args.a_scales, args.w_scales[0], args.y[0], p.M, static_cast<int>(p.N), p.split, stream));
}

// The activations as codes at the start of the workspace, unless the kernel quantizes them.
int quantize_into(const Sizes& d, const Product& p, const uint16_t* x, void* workspace, W8TileArgs& args, hipStream_t stream) {
    if (p.quantize) {
        args.x = x;
        return W4A16_OK;
    }
    int8_t* codes = static_cast<int8_t*>(workspace);
    float* scales = static_cast<float*>(after(workspace, round256(static_cast<uint64_t>(d.T) * d.K)));
    args.a = codes;
    args.a_scales = scales;
    return to_status(launch_w8_quantize(x, false, codes, scales, d.T, static_cast<int>(d.K), stream));
}

// Gradient rows [R, N] as 16-byte rows: themselves, or their padded copy.
int pad_gradient(const uint16_t* dy, const Sizes& d, void* copy, hipStream_t stream, const uint16_t** rows) {
    *rows = dy;
    if (d.N % 8 == 0) return W4A16_OK;
    *rows = static_cast<uint16_t*>(copy);
    return to_status(launch_mx_pad_rows(dy, static_cast<uint16_t*>(copy), d.R, static_cast<int>(d.N), stream));
}

int run_columns(const Product& p, W8ColumnsArgs& args, const Sizes& d, void* partials, hipStream_t stream) {
    args.E = static_cast<int>(d.E);
    args.R = static_cast<int>(d.R);
    args.N = static_cast<int>(d.N);
    args.K = static_cast<int>(d.K);
    args.pitch = static_cast<int>(padded(d.N));
    args.split = p.split;
    args.height = p.height;
    args.cut = p.cut;
    args.cus = p.cus;
    args.ws = static_cast<float*>(partials);
    const hipError_t e = launch_w8_columns(p.tile, args, stream);
    if (e != hipSuccess || p.split == 1) return to_status(e);
    return to_status(launch_mx_sum(args.ws, args.y, 1, p.M * p.N, p.split, stream));
}

uint64_t weight_bytes(const Sizes& d) { return static_cast<uint64_t>(d.E) * d.N * d.K; }
uint64_t scale_bytes(const Sizes& d) { return static_cast<uint64_t>(d.E) * d.N * 4; }
uint64_t row_bytes(int64_t R, int64_t N) { return static_cast<uint64_t>(R) * N * 2; }

// Checks of the routing of an experts' call.
int check_routing(const Sizes& d, const int32_t* offsets, const int32_t* tokens, bool gathers) {
    if (!offsets) return W4A16_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(tokens, 4)) return W4A16_ERR_ALIGN;
    if (!gathers) return W4A16_OK;
    // gathered rows are addressed by 32-bit offsets into the codes
    if (tokens ? d.T * d.K > kMaxDim : d.T != d.R) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int run_forward_call(int32_t op, const Sizes& d, const uint16_t* x, const int8_t* codes, const float* scales,
                     const int32_t* offsets, const int32_t* tokens, uint16_t* y, int32_t split_k, void* workspace,
                     size_t workspace_bytes, void* stream) {
    int st = check_sizes(op, d, split_k);
    if (st != W4A16_OK) return st;
    if (!x || !y) return W4A16_ERR_NULL;
    st = check_weights(codes, scales);
    if (st == W4A16_OK && has_experts(op)) st = check_routing(d, offsets, tokens, true);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(y, 2)) return W4A16_ERR_ALIGN;
    if (!disjoint({{y, row_bytes(d.R, d.N)}},
                  {{x, row_bytes(d.T, d.K)}, {codes, weight_bytes(d)}, {scales, scale_bytes(d)},
                   {offsets, 4 * static_cast<uint64_t>(d.E + 1)}, {tokens, 4 * static_cast<uint64_t>(d.R)}}))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(op, d, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    W8TileArgs args = tile_args(d, p, offsets, tokens, y);
    args.w[0] = codes;
    args.w_scales[0] = scales;
    st = quantize_into(d, p, x, workspace, args, s);
    if (st != W4A16_OK) return st;
    return run_forward(W8Epilogue::kStore, p, args, after(workspace, fixed_bytes(op, d, p)), s);
}

int run_backward_call(int32_t op, const Sizes& d, const uint16_t* dy, const int8_t* codes, const float* scales,
                      const int32_t* offsets, uint16_t* dx, int32_t split_k, void* workspace, size_t workspace_bytes,
                      void* stream) {
    int st = check_sizes(op, d, split_k);
    if (st != W4A16_OK) return st;
    if (!dy || !dx) return W4A16_ERR_NULL;
    st = check_weights(codes, scales);
    if (st == W4A16_OK && has_experts(op)) st = check_routing(d, offsets, nullptr, false);
    if (st != W4A16_OK) return st;
    if (!aligned(dy, 16) || !aligned(dx, 2)) return W4A16_ERR_ALIGN;
    if (!disjoint({{dx, row_bytes(d.R, d.K)}}, {{dy, row_bytes(d.R, d.N)}, {codes, weight_bytes(d)}, {scales, scale_bytes(d)},
                                               {offsets, 4 * static_cast<uint64_t>(d.E + 1)}}))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(op, d, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    W8ColumnsArgs args{};
    st = pad_gradient(dy, d, workspace, s, &args.g[0]);
    if (st != W4A16_OK) return st;
    args.w[0] = codes;
    args.w_scales[0] = scales;
    args.y = dx;
    args.offsets = offsets;
    args.sets = 1;
    return run_columns(p, args, d, after(workspace, fixed_bytes(op, d, p)), s);
}

int check_route(int64_t T, int64_t E, int64_t top_k) {
    if (T < 1 || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > E) return W4A16_ERR_SHAPE;
    return T > kMaxTokens || T * top_k > kMaxRows ? W4A16_ERR_SHAPE : W4A16_OK;
}

int check_logits(const void* logits, int32_t type) {
    if (type != W8A8_BF16 && type != W8A8_FP32) return W4A16_ERR_UNSUPPORTED;
    if (!logits) return W4A16_ERR_NULL;
    return aligned(logits, type == W8A8_FP32 ? 4 : 2) ? W4A16_OK : W4A16_ERR_ALIGN;
}

int check_combine(int64_t T, int64_t top_k, int64_t R, int64_t N, bool backward) {
    if (T < 1 || T > kMaxTokens || top_k < 1 || top_k > kMaxTopK || R < 1 || R > kMaxRows || N < 1 || N > kMaxRows)
        return W4A16_ERR_SHAPE;
    // a wave per token and expert backward, a thread per eight columns forward
    const bool fits = backward ? T * top_k <= kMaxThreads / 64 - 4 : T * ceil_div(N, 8) <= kMaxThreads - 256;
    return fits && T * top_k <= kMaxRows ? W4A16_OK : W4A16_ERR_SHAPE;
}

}  // namespace

extern "C" {

int w8a8_quantize_rows(const void* x, int32_t x_type, int8_t* codes, float* scales, int64_t R, int64_t K, void* stream) {
    const int st = check_matrix(R, K);
    if (st != W4A16_OK) return st;
    if (x_type != W8A8_BF16 && x_type != W8A8_FP32) return W4A16_ERR_UNSUPPORTED;
    if (!x || !codes || !scales) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return W4A16_ERR_ALIGN;
    const uint64_t n = static_cast<uint64_t>(R) * K;
    if (!disjoint({{codes, n}, {scales, 4 * static_cast<uint64_t>(R)}}, {{x, n * (x_type == W8A8_FP32 ? 4 : 2)}}))
        return W4A16_ERR_OVERLAP;
    return to_status(launch_w8_quantize(x, x_type == W8A8_FP32, codes, scales, R, static_cast<int>(K), static_cast<hipStream_t>(stream)));
}

int w8a8_plan(int32_t op, int64_t E, int64_t T, int64_t R, int64_t N, int64_t K, int32_t split_k, int32_t num_cus,
              w4a16_plan_t* out) {
    if (!out) return W4A16_ERR_NULL;
    const Sizes d{E, T, R, N, K};
    Product p;
    int32_t cus;
    const int st = plan_call(op, d, split_k, num_cus, &p, &cus);
    if (st != W4A16_OK) return st;
    const bool back = is_backward(op);
    const W8TileShape& s = back ? kW8ColumnTiles[p.tile] : kW8Tiles[p.tile];
    out->path = W4A16_PATH_W8A8;
    out->tile_m = p.height;
    out->tile_n = !back && is_gated(op) ? s.bn / 2 : s.bn;
    out->tile_k = back ? kW8ColumnStep : kW8Step;
    out->block_threads = 64 * s.waves;
    out->k_waves = 1;
    out->variant = p.tile + (!has_experts(op) && p.cut > 1 ? 10 : 0);
    if (p.decode) {
        out->path = W4A16_PATH_W8A8_QMV;
        out->tile_m = p.qmv.rows;
        out->tile_n = kW8QmvColumns;
        out->tile_k = kW8Step;
        out->block_threads = 64 * p.qmv.waves;
        out->k_waves = p.qmv.waves;
        out->variant = p.quantize;
    }
    out->grid_x = static_cast<int32_t>(ceil_div(p.N, out->tile_n));
    out->grid_y = static_cast<int32_t>(row_blocks(d, has_experts(op), out->tile_m));
    out->grid_z = p.split;
    out->split_k = p.split;
    out->num_cus = cus;
    out->workspace_bytes = fixed_bytes(op, d, p) + partial_bytes(p);
    return W4A16_OK;
}

int qmm_w8a8(const int8_t* xq, const float* xs, const int8_t* codes, const float* scales, uint16_t* y, int64_t M, int64_t N,
             int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    const Sizes d{1, M, M, N, K};
    int st = check_sizes(W8A8_QMM, d, split_k);
    if (st != W4A16_OK) return st;
    st = check_weights(xq, xs);
    if (st == W4A16_OK) st = check_weights(codes, scales);
    if (st != W4A16_OK) return st;
    if (!y) return W4A16_ERR_NULL;
    if (!aligned(y, 2)) return W4A16_ERR_ALIGN;
    if (!disjoint({{y, row_bytes(M, N)}}, {{xq, static_cast<uint64_t>(M) * K}, {xs, 4 * static_cast<uint64_t>(M)},
                                           {codes, weight_bytes(d)}, {scales, scale_bytes(d)}}))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(W8A8_QMM, d, split_k, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    W8TileArgs args = tile_args(d, p, nullptr, nullptr, y);
    args.a = xq;
    args.a_scales = xs;
    args.w[0] = codes;
    args.w_scales[0] = scales;
    return run_forward(W8Epilogue::kStore, p, args, workspace, static_cast<hipStream_t>(stream));
}

int w8a8_linear(const uint16_t* x, const int8_t* codes, const float* scales, uint16_t* y, int64_t M, int64_t N, int64_t K,
                int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    return run_forward_call(W8A8_LINEAR, Sizes{1, M, M, N, K}, x, codes, scales, nullptr, nullptr, y, split_k, workspace,
                            workspace_bytes, stream);
}

int w8a8_linear_backward(const uint16_t* dy, const int8_t* codes, const float* scales, uint16_t* dx, int64_t M, int64_t N,
                         int64_t K, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream) {
    return run_backward_call(W8A8_LINEAR_BACKWARD, Sizes{1, M, M, N, K}, dy, codes, scales, nullptr, dx, split_k, workspace,
                             workspace_bytes, stream);
}

int w8a8_experts_linear(const uint16_t* x, const int8_t* codes, const float* scales, const int32_t* offsets,
                        const int32_t* tokens, uint16_t* y, int64_t E, int64_t T, int64_t R, int64_t N, int64_t K,
                        void* workspace, size_t workspace_bytes, void* stream) {
    return run_forward_call(W8A8_EXPERTS_LINEAR, Sizes{E, T, R, N, K}, x, codes, scales, offsets, tokens, y, 0, workspace,
                            workspace_bytes, stream);
}

int w8a8_experts_linear_backward(const uint16_t* dy, const int8_t* codes, const float* scales, const int32_t* offsets,
                                 uint16_t* dx, int64_t E, int64_t R, int64_t N, int64_t K, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    return run_backward_call(W8A8_EXPERTS_LINEAR_BACKWARD, Sizes{E, R, R, N, K}, dy, codes, scales, offsets, dx, 0,
                             workspace, workspace_bytes, stream);
}

int w8a8_experts_gate_up_swiglu(const uint16_t* x, const int8_t* codes_gate, const float* scales_gate,
                                const int8_t* codes_up, const float* scales_up, const int32_t* offsets,
                                const int32_t* tokens, uint16_t* h, int64_t E, int64_t T, int64_t R, int64_t N, int64_t K,
                                void* workspace, size_t workspace_bytes, void* stream) {
    const Sizes d{E, T, R, N, K};
    int st = check_sizes(W8A8_EXPERTS_GATE_UP, d, 0);
    if (st != W4A16_OK) return st;
    if (!x || !h) return W4A16_ERR_NULL;
    st = check_weights(codes_gate, scales_gate);
    if (st == W4A16_OK) st = check_weights(codes_up, scales_up);
    if (st == W4A16_OK) st = check_routing(d, offsets, tokens, true);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(h, 2)) return W4A16_ERR_ALIGN;
    if (!disjoint({{h, row_bytes(R, N)}},
                  {{x, row_bytes(T, K)}, {codes_gate, weight_bytes(d)}, {scales_gate, scale_bytes(d)},
                   {codes_up, weight_bytes(d)}, {scales_up, scale_bytes(d)}, {offsets, 4 * static_cast<uint64_t>(E + 1)},
                   {tokens, 4 * static_cast<uint64_t>(R)}}))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(W8A8_EXPERTS_GATE_UP, d, 0, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    W8TileArgs args = tile_args(d, p, offsets, tokens, h);
    args.w[0] = codes_gate;
    args.w[1] = codes_up;
    args.w_scales[0] = scales_gate;
    args.w_scales[1] = scales_up;
    st = quantize_into(d, p, x, workspace, args, s);
    if (st != W4A16_OK) return st;
    return run_forward(W8Epilogue::kGlu, p, args, nullptr, s);
}

int w8a8_experts_gate_up_swiglu_backward(const uint16_t* x, const int8_t* codes_gate, const float* scales_gate,
                                         const int8_t* codes_up, const float* scales_up, const uint16_t* dh,
                                         const int32_t* offsets, const int32_t* tokens, uint16_t* dx, uint16_t* dgate,
                                         uint16_t* dup, int64_t E, int64_t T, int64_t R, int64_t N, int64_t K,
                                         void* workspace, size_t workspace_bytes, void* stream) {
    const Sizes d{E, T, R, N, K};
    const int32_t op = W8A8_EXPERTS_GATE_UP_BACKWARD;
    int st = check_sizes(op, d, 0);
    if (st != W4A16_OK) return st;
    if (!x || !dh || !dx || !dgate || !dup) return W4A16_ERR_NULL;
    st = check_weights(codes_gate, scales_gate);
    if (st == W4A16_OK) st = check_weights(codes_up, scales_up);
    if (st == W4A16_OK) st = check_routing(d, offsets, tokens, true);
    if (st != W4A16_OK) return st;
    if (!aligned(x, 16) || !aligned(dgate, 2) || !aligned(dup, 2) || !aligned(dh, 2) || !aligned(dx, 2))
        return W4A16_ERR_ALIGN;
    if (!disjoint({{dx, row_bytes(R, K)}, {dgate, row_bytes(R, N)}, {dup, row_bytes(R, N)}},
                  {{x, row_bytes(T, K)}, {dh, row_bytes(R, N)}, {codes_gate, weight_bytes(d)}, {scales_gate, scale_bytes(d)},
                   {codes_up, weight_bytes(d)}, {scales_up, scale_bytes(d)}, {offsets, 4 * static_cast<uint64_t>(E + 1)},
                   {tokens, 4 * static_cast<uint64_t>(R)}}))
        return W4A16_ERR_OVERLAP;
    Product p;
    st = fit(op, d, 0, workspace, workspace_bytes, &p);
    if (st != W4A16_OK) return st;
    int32_t cus;
    st = query_num_cus(&cus);
    if (st != W4A16_OK) return st;
    const Product again = both_again(d, cus);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    W8TileArgs args = tile_args(d, again, offsets, tokens, dgate);
    args.w[0] = codes_gate;
    args.w[1] = codes_up;
    args.w_scales[0] = scales_gate;
    args.w_scales[1] = scales_up;
    args.dh = dh;
    args.y[1] = dup;
    void* gradients = after(workspace, activation_bytes(d));
    args.scaled[0] = static_cast<uint16_t*>(gradients);
    args.scaled[1] = static_cast<uint16_t*>(after(gradients, gradient_bytes(op, d) / 2));
    st = quantize_into(d, again, x, workspace, args, s);
    if (st == W4A16_OK) st = run_forward(W8Epilogue::kGluGrad, again, args, nullptr, s);
    if (st != W4A16_OK) return st;
    W8ColumnsArgs columns{};
    columns.g[0] = args.scaled[0];
    columns.g[1] = args.scaled[1];
    columns.w[0] = codes_gate;
    columns.w[1] = codes_up;
    columns.y = dx;
    columns.offsets = offsets;
    columns.sets = 2;
    return run_columns(p, columns, d, nullptr, s);
}

uint64_t experts_route_workspace_bytes(int64_t T, int64_t E) {
    if (check_route(T, E, 1) != W4A16_OK) return 0;
    return experts_route_bytes(T, static_cast<int>(E));
}

int experts_route(const void* logits, int32_t type, float* weights, int32_t* experts, int32_t* positions, int32_t* tokens,
                  int32_t* offsets, int64_t T, int64_t E, int32_t top_k, int32_t renormalize, void* workspace,
                  size_t workspace_bytes, void* stream) {
    int st = check_route(T, E, top_k);
    if (st == W4A16_OK) st = check_logits(logits, type);
    if (st != W4A16_OK) return st;
    if (!weights || !experts || !positions || !tokens || !offsets) return W4A16_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(experts, 4) || !aligned(positions, 4) || !aligned(tokens, 4) || !aligned(offsets, 4))
        return W4A16_ERR_ALIGN;
    const uint64_t n = 4 * static_cast<uint64_t>(T) * top_k;
    if (!disjoint({{weights, n}, {experts, n}, {positions, n}, {tokens, n}, {offsets, 4 * static_cast<uint64_t>(E + 1)}},
                  {{logits, static_cast<uint64_t>(T) * E * (type == W8A8_FP32 ? 4 : 2)}}))
        return W4A16_ERR_OVERLAP;
    const uint64_t need = experts_route_bytes(T, static_cast<int>(E));
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return W4A16_ERR_ALIGN;
    return to_status(launch_experts_route(logits, type == W8A8_FP32, top_k, renormalize != 0, weights, experts, positions, tokens,
                                          offsets, T, static_cast<int>(E), need > 0 ? static_cast<int*>(workspace) : nullptr,
                                          static_cast<hipStream_t>(stream)));
}

int experts_route_backward(const void* logits, int32_t type, const int32_t* experts, const float* dweights, void* dlogits,
                           int64_t T, int64_t E, int32_t top_k, int32_t renormalize, void* stream) {
    int st = check_route(T, E, top_k);
    if (st == W4A16_OK) st = check_logits(logits, type);
    if (st != W4A16_OK) return st;
    if (!experts || !dweights || !dlogits) return W4A16_ERR_NULL;
    if (!aligned(experts, 4) || !aligned(dweights, 4) || !aligned(dlogits, type == W8A8_FP32 ? 4 : 2)) return W4A16_ERR_ALIGN;
    const uint64_t n = 4 * static_cast<uint64_t>(T) * top_k, size = static_cast<uint64_t>(T) * E * (type == W8A8_FP32 ? 4 : 2);
    if (!disjoint({{dlogits, size}}, {{logits, size}, {experts, n}, {dweights, n}})) return W4A16_ERR_OVERLAP;
    return to_status(launch_experts_route_backward(logits, type == W8A8_FP32, experts, dweights, dlogits, T, static_cast<int>(E),
                                                   top_k, renormalize != 0, static_cast<hipStream_t>(stream)));
}

int experts_combine(const uint16_t* y, const int32_t* positions, const float* weights, uint16_t* out, int64_t T, int32_t top_k,
                    int64_t R, int64_t N, void* stream) {
    const int st = check_combine(T, top_k, R, N, false);
    if (st != W4A16_OK) return st;
    if (!y || !positions || !out) return W4A16_ERR_NULL;
    if (!aligned(y, 2) || !aligned(out, 2) || !aligned(positions, 4) || !aligned(weights, 4)) return W4A16_ERR_ALIGN;
    const uint64_t n = 4 * static_cast<uint64_t>(T) * top_k;
    if (!disjoint({{out, row_bytes(T, N)}}, {{y, row_bytes(R, N)}, {positions, n}, {weights, n}})) return W4A16_ERR_OVERLAP;
    return to_status(launch_experts_combine(y, positions, weights, out, T, top_k, R, static_cast<int>(N), static_cast<hipStream_t>(stream)));
}

int experts_combine_backward(const uint16_t* dout, const uint16_t* y, const int32_t* positions, const float* weights,
                             uint16_t* dy, float* dweights, int64_t T, int32_t top_k, int64_t R, int64_t N, void* stream) {
    const int st = check_combine(T, top_k, R, N, true);
    if (st != W4A16_OK) return st;
    if (!dout || !y || !positions || !weights || !dy || !dweights) return W4A16_ERR_NULL;
    if (!aligned(dout, 2) || !aligned(y, 2) || !aligned(dy, 2) || !aligned(positions, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return W4A16_ERR_ALIGN;
    const uint64_t n = 4 * static_cast<uint64_t>(T) * top_k, rows = row_bytes(R, N);
    if (!disjoint({{dy, rows}, {dweights, n}}, {{dout, row_bytes(T, N)}, {y, rows}, {positions, n}, {weights, n}}))
        return W4A16_ERR_OVERLAP;
    return to_status(launch_experts_combine_backward(dout, y, positions, weights, dy, dweights, T, top_k, R, static_cast<int>(N),
                                                     static_cast<hipStream_t>(stream)));
}

}  // extern "C"
