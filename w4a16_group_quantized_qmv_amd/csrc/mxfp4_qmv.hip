// MXFP4 products for decode rows (M <= 16): the weight-only projection, the product of two MXFP4
// operands, and the gated pair.
//
//   y[m, n] = sum_k x[m, k] w[n, k]         h[m, n] = silu(g[m, n]) u[m, n]
//
// Bound by memory: every weight byte is read once (0.53 bytes a value) and does 2 M operations a
// value, far below the matrix cores' ratio.  So the whole matrix has to be requested within about
// one memory latency:
//  * A unit is 1 KB of codes, one block (16 bytes) per lane: C columns x S * 128 values, S C = 16.  The
//    16 x 16 MFMA takes S slices of C columns as its 16 rows and S slices of ROWS <= C activation rows
//    as its 16 columns; of the products of different slices, which are computed as well, nothing is
//    kept.  Few rows (S = 4) thus give small workgroups of 4 columns, many of them, and reads of 256
//    consecutive bytes.
//  * A workgroup has C columns; its waves take consecutive shares of the contraction.  A wave issues
//    every load of up to UB units (codes, scales, activations) before it uses the first.
//  * bf16 activations go through a slice of LDS of the wave's own: they are loaded 16 consecutive
//    bytes per lane and read back 64 bytes per lane as the blocks lie, chunk c of MFMA column r at
//    c ^ r, so that 16 columns' reads fall into 16 bank groups.
//  * The waves' sums and the slices' are added in order by the first threads.
#include "mxfp4_device.h"
#include "mxfp4_internal.h"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr uint32_t kOutside = 0x80000000u;   // a buffer offset that no resource here reaches

__device__ __forceinline__ __amdgpu_buffer_rsrc_t qmv_resource(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFFll ? 0x7FFFFFFFll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(n), 0x00020000);
}

// ROWS: activation rows that an instance holds (1, 2, 4, 8 or 16); NP: weight sets; UB: units in flight.
template <bool CODES, int ROWS, int NP, int UB>
__global__ __launch_bounds__(1024) void mx_qmv_kernel(const MxTileArgs p, int share) {
    constexpr int S = ROWS <= 4 ? 4 : 16 / ROWS, C = 16 / S;
    constexpr int XL = CODES ? 1 : (ROWS * S + 3) / 4;        // activation loads of a unit
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int r = lane & 15, q = lane >> 4, slice = r / C, rc = r % C;
    const int c0 = blockIdx.x * C;
    const int blocks = p.L / kMxBlock, row_codes = blocks * 16;
    const int units = (blocks + 4 * S - 1) / (4 * S);
    const int u_begin = wave * share, u_end = min(units, u_begin + share);

    const int64_t columns = p.N - c0;
    __amdgpu_buffer_rsrc_t cr[NP], sr[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        cr[s] = qmv_resource(p.w[s] + static_cast<int64_t>(c0) * row_codes, columns * row_codes);
        sr[s] = qmv_resource(p.w_scales[s] + static_cast<int64_t>(c0) * blocks, columns * blocks);
    }
    const __amdgpu_buffer_rsrc_t xr = qmv_resource(p.a[0], static_cast<int64_t>(p.M) * p.pitch);
    const __amdgpu_buffer_rsrc_t xsr = qmv_resource(p.a_scales, CODES ? static_cast<int64_t>(p.M) * blocks : 0);
    const int own_block = 4 * slice + q;                      // this lane's block of a unit

    f32x4_t acc[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) acc[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint8_t* xs = lds + wave * (ROWS * S * 256);

    for (int u0 = u_begin; u0 < u_end; u0 += UB) {
        u32x4_t codes[UB][NP], xv[UB][XL];
        uint32_t scale[UB][NP], xscale[UB];
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int b = 4 * S * (u0 + i) + own_block;
            const bool inside = u0 + i < u_end && b < blocks;
#pragma unroll
            for (int s = 0; s < NP; ++s) {
                const uint32_t co = inside ? static_cast<uint32_t>(rc * row_codes + 16 * b) : kOutside;
                codes[i][s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(cr[s], co, 0, kStreamedOnce));
                const uint32_t so = inside ? static_cast<uint32_t>(rc * blocks + b) : kOutside;
                scale[i][s] = __builtin_amdgcn_raw_buffer_load_b8(sr[s], so, 0, 0);
            }
            if constexpr (CODES) {
                const uint32_t xo = inside ? static_cast<uint32_t>(rc * row_codes + 16 * b) : kOutside;
                xv[i][0] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, xo, 0, 0));
                const uint32_t xso = inside ? static_cast<uint32_t>(rc * blocks + b) : kOutside;
                xscale[i] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso, 0, 0);
            } else {
                // piece t of the unit: 16 bytes of row t / (16 S), rows of 16 S pieces
#pragma unroll
                for (int j = 0; j < XL; ++j) {
                    const int t = 64 * j + lane, m = t / (16 * S), piece = t % (16 * S);
                    const int k = 128 * S * (u0 + i) + 8 * piece;
                    const bool in = u0 + i < u_end && m < min(ROWS, p.M) && k < p.L;
                    const uint32_t xo = in ? static_cast<uint32_t>(m * p.pitch + 2 * k) : kOutside;
                    xv[i][j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(xr, xo, 0, 0));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            if constexpr (CODES) {
#pragma unroll
                for (int s = 0; s < NP; ++s)
                    acc[s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        mx_operand(codes[i][s]), mx_operand(xv[i][0]), acc[s], 4, 4, 0, static_cast<int>(scale[i][s]), 0,
                        static_cast<int>(xscale[i]));
            } else {
#pragma unroll
                for (int j = 0; j < XL; ++j) {
                    const int t = 64 * j + lane, m = t / (16 * S), piece = t % (16 * S);
                    // MFMA column of the piece: its slice's row m
                    const int col = (piece >> 4) * C + m;
                    if (ROWS * S >= 4 || t < ROWS * S * 16)
                        *reinterpret_cast<u32x4_t*>(xs + (m * S + (piece >> 4)) * 256 + 16 * ((piece ^ col) & 15)) = xv[i][j];
                }
                wave_lds_fence();
                const int m = min(rc, ROWS - 1), col = slice * C + m;
                const uint8_t* row = xs + (m * S + slice) * 256;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(row + 16 * (((4 * q + j) ^ col) & 15));
#pragma unroll
                    for (int s = 0; s < NP; ++s)
                        acc[s] = mfma16x16x32(
                            __builtin_bit_cast(bf16x8_t, mx_decode_word(codes[i][s][j], mx_scale(scale[i][s]))),
                            __builtin_bit_cast(bf16x8_t, x), acc[s]);
                }
                if (i + 1 < UB || u0 + UB < u_end) wave_lds_fence();
            }
        }
    }

    // register e of lane l: weight row 4 (l / 16) + e, activation column l % 16; wanted where both are
    // of one slice
    __syncthreads();
    float* sums = reinterpret_cast<float*>(lds);              // [set][wave][slice][row][column]
    const int w_slice = 4 * q / C, w_col = 4 * q % C;
    if (w_slice == slice) {
#pragma unroll
        for (int s = 0; s < NP; ++s)
            *reinterpret_cast<f32x4_t*>(sums + ((s * waves + wave) * S + slice) * C * C + rc * C + w_col) = acc[s];
    }
    __syncthreads();
    for (int t = threadIdx.x; t < C * C; t += blockDim.x) {
        const int m = t / C, n = c0 + t % C;
        if (m >= p.M || n >= p.N) continue;
        float v[NP];
#pragma unroll
        for (int s = 0; s < NP; ++s) {
            v[s] = 0.f;
            for (int w = 0; w < waves * S; ++w) v[s] += sums[(s * waves * S + w) * C * C + t];
        }
        if constexpr (NP == 2) v[0] = v[0] * mx_sigmoid(v[0]) * v[1];
        p.y[0][static_cast<size_t>(m) * p.N + n] = f32_to_bf16_bits(v[0]);
    }
}

}  // namespace

bool mx_qmv_shape(MxOperands op, int sets, int M, int K, MxQmvShape* out) {
    if (M > kMxQmvRows || op == MxOperands::kColumns) return false;
    const bool codes = op == MxOperands::kCodes;
    out->rows = M <= 1 && !codes ? 1 : M <= 2 && !codes ? 2 : M <= 4 ? 4 : M <= 8 ? 8 : 16;
    const int S = out->rows <= 4 ? 4 : 16 / out->rows;
    out->columns = 16 / S;
    const int units = (K / kMxBlock + 4 * S - 1) / (4 * S);
    out->share = (units + kMxQmvWaves - 1) / kMxQmvWaves;
    out->waves = (units + out->share - 1) / out->share;
    out->batch = out->share == 1 ? 1 : out->share == 2 ? 2 : 4;
    const size_t x = codes ? 0 : static_cast<size_t>(out->rows) * S * 256 * out->waves;
    const size_t sums = static_cast<size_t>(sets) * out->waves * S * out->columns * out->columns * sizeof(float);
    out->lds = std::max(x, sums);
    return true;
}

hipError_t launch_mx_qmv(MxOperands op, MxEpilogue epi, const MxTileArgs& args, hipStream_t stream) {
    MxQmvShape s;
    const int sets = epi == MxEpilogue::kGlu ? 2 : 1;
    if (!mx_qmv_shape(op, sets, args.M, args.L, &s)) return hipErrorInvalidValue;
    const dim3 grid((args.N + s.columns - 1) / s.columns), block(64 * s.waves);
    auto run = [&](auto kernel) {
        W4A16_LAUNCH(kernel, grid, block, s.lds, stream, args, s.share);
        return hipGetLastError();
    };
    auto batched = [&](auto cc, auto rc, auto nc) {
        constexpr bool codes = decltype(cc)::value;
        constexpr int rows = decltype(rc)::value, np = decltype(nc)::value;
        if (s.batch == 1) return run(mx_qmv_kernel<codes, rows, np, 1>);
        if (s.batch == 2) return run(mx_qmv_kernel<codes, rows, np, 2>);
        return run(mx_qmv_kernel<codes, rows, np, 4>);
    };
    auto sized = [&](auto cc, auto nc) {
        if constexpr (!decltype(cc)::value) {
            if (s.rows == 1) return batched(cc, std::integral_constant<int, 1>{}, nc);
            if (s.rows == 2) return batched(cc, std::integral_constant<int, 2>{}, nc);
        }
        if (s.rows == 4) return batched(cc, std::integral_constant<int, 4>{}, nc);
        if (s.rows == 8) return batched(cc, std::integral_constant<int, 8>{}, nc);
        return batched(cc, std::integral_constant<int, 16>{}, nc);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (op == MxOperands::kCodes) return sized(std::true_type{}, One{});
    return sets == 2 ? sized(std::false_type{}, Two{}) : sized(std::false_type{}, One{});
}

}  // namespace w4a16
