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
// Measured on MI355X in a graph, the same weights again (in the last-level cache where they fit) / in turn
// with copies of 512 MB and more, us: one row of 9728 x 2560 (2560 values) 5.1 / 5.7 (2.3 TB/s), 8 rows
// 7.9 / 8.1, 16 rows 9.5 / 10.1; the gated pair, one row 8.3 / 8.7 (3.0 TB/s); one row of 9728 x 9728
// 12.5 / 14.0 (3.6 TB/s); five rows of 151936 x 2560 in the wide form 39 / 41 (5.0 TB/s).  Small matrices
// are a few memory latencies, whatever their bytes.
#include "mxfp4_device.h"
#include "mxfp4_internal.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

// Activations of the decode kernels.
enum class MxX { kBf16, kCodes, kQuantize };   // as they are, MXFP4, or bf16 quantized to MXFP4 on the way

// A lane's block of 32 bf16 values, in order, as an MXFP4 operand and its scale byte (the rule of
// mx_quantize_kernel).
__device__ __forceinline__ u32x4_t quantize_block(const u32x4_t (&v)[4], uint32_t& e) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t top = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[j][i] & 0x7FFF7FFFu));
    const uint32_t field = static_cast<uint32_t>(max(top[0], top[1])) >> 7;
    e = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
    const float scale = mx_scale(e);
    u32x4_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // (through locals: a vector element as the operand of a bit cast stands for element 0)
        const uint32_t v0 = v[j][0], v1 = v[j][1], v2 = v[j][2], v3 = v[j][3];
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v0), scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v1), scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v2), scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v3), scale, 3);
        r[j] = e == 255u ? 0u : w;
    }
    return r;
}

__device__ __forceinline__ f32x4_t mx_mfma16(const u32x4_t& a, uint32_t sa, const u32x4_t& b, uint32_t sb,
                                             const f32x4_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, 0,
                                                            static_cast<int>(sa), 0, static_cast<int>(sb));
}

// ROWS: activation rows that an instance holds (1, 2, 4, 8 or 16); NP: weight sets; UB: units in flight.
template <MxX X, int ROWS, int NP, int UB>
__global__ __launch_bounds__(1024) void mx_qmv_kernel(const MxTileArgs p, int share) {
    constexpr int S = ROWS <= 4 ? 4 : 16 / ROWS, C = 16 / S;
    constexpr bool CODES = X == MxX::kCodes;
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
        cr[s] = mx_resource(p.w[s] + static_cast<int64_t>(c0) * row_codes, columns * row_codes);
        sr[s] = mx_resource(p.w_scales[s] + static_cast<int64_t>(c0) * blocks, columns * blocks);
    }
    const __amdgpu_buffer_rsrc_t xr = mx_resource(p.a[0], static_cast<int64_t>(p.M) * p.pitch);
    const __amdgpu_buffer_rsrc_t xsr = mx_resource(p.a_scales, CODES ? static_cast<int64_t>(p.M) * blocks : 0);
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
                for (int s = 0; s < NP; ++s) acc[s] = mx_mfma16(codes[i][s], scale[i][s], xv[i][0], xscale[i], acc[s]);
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
                u32x4_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const u32x4_t*>(row + 16 * (((4 * q + j) ^ col) & 15));
                if constexpr (X == MxX::kQuantize) {
                    uint32_t e;
                    const u32x4_t xq = quantize_block(x, e);
#pragma unroll
                    for (int s = 0; s < NP; ++s) acc[s] = mx_mfma16(codes[i][s], scale[i][s], xq, e, acc[s]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int s = 0; s < NP; ++s)
                            acc[s] = mfma16x16x32(
                                __builtin_bit_cast(bf16x8_t, mx_decode_word(codes[i][s][j], mx_scale(scale[i][s]))),
                                __builtin_bit_cast(bf16x8_t, x[j]), acc[s]);
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

// `into` with lanes 8 .. 15 (BANKS 0xC) or 0 .. 7 (0x3) of every sixteen replaced by the other eight
// lanes of `from` (DPP row_ror:8).
template <int BANKS>
__device__ __forceinline__ uint32_t half_row_move(uint32_t into, uint32_t from) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(static_cast<int>(into), static_cast<int>(from), 0x128, 0xF, BANKS, false));
}

// The wide form: many columns (a vocabulary head).  A wave streams whole blocks of 16 columns, S = 1,
// a window of 512 values (256 consecutive bytes of each column and its 16 scale bytes) at a time with
// the next window in flight; the activations are staged once per workgroup, which takes blocks until
// none is left.  A load takes 128 bytes of eight columns rather than 64 of sixteen: half lines
// streamed past the cache measured 48.5 us against 41 on the 151936 x 2560 head, and 8 lane moves
// per 2 KB put the blocks where the matrix instruction wants them.  K is a multiple of 512 and the scale rows are 16-byte aligned.
// (Two weight sets in turn, for the gated pair, measured 17 us against the other form's 9 to 12 on 9728
// columns and as much on 16384.)
template <MxX X>
__global__ __launch_bounds__(64 * kMxWideWaves) void mx_qmv_wide_kernel(const MxTileArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int blocks = p.L / kMxBlock, row_codes = blocks * 16, windows = blocks / 16;
    const int first = (blockIdx.x * kMxWideWaves + wave), stride = gridDim.x * kMxWideWaves;
    const int column_blocks = (p.N + 15) / 16;

    // x in LDS.  kBf16: rows of 2 K bytes, 16-byte chunk c of row m at c ^ m (the low four bits).
    // Else codes, rows of K / 2 bytes with chunk c at c ^ m, and then scale rows of K / 32 bytes.
    const int rows = p.M;
    const int x_pitch = X == MxX::kBf16 ? 2 * p.L : p.L / 2;
    uint8_t* xs_scale = lds + rows * x_pitch;
    if constexpr (X == MxX::kBf16) {
        const int chunks = p.L / 8;
        for (int t = threadIdx.x; t < rows * chunks; t += 64 * kMxWideWaves) {
            const int m = t / chunks, c = t - m * chunks;
            *reinterpret_cast<u32x4_t*>(lds + m * x_pitch + 16 * (c ^ m)) =
                load16(static_cast<const uint8_t*>(p.a[0]) + m * p.pitch + 16 * c);
        }
    } else {
        for (int t = threadIdx.x; t < rows * blocks; t += 64 * kMxWideWaves) {
            const int m = t / blocks, c = t - m * blocks;
            u32x4_t v;
            uint32_t e;
            if constexpr (X == MxX::kCodes) {
                v = load16(static_cast<const uint8_t*>(p.a[0]) + m * p.pitch + 16 * c);
                e = p.a_scales[m * blocks + c];
            } else {
                u32x4_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = load16(static_cast<const uint8_t*>(p.a[0]) + m * p.pitch + 64 * c + 16 * j);
                v = quantize_block(x, e);
            }
            *reinterpret_cast<u32x4_t*>(lds + m * x_pitch + 16 * (c ^ m)) = v;
            xs_scale[m * blocks + c] = static_cast<uint8_t>(e);
        }
    }
    __syncthreads();

    u32x4_t codes[2][4], scales[2];
    auto load = [&](int block, int window, auto ic) {
        constexpr int par = decltype(ic)::value;
        const int64_t c0 = 16 * static_cast<int64_t>(block), left = block < column_blocks ? p.N - c0 : 0;
        const __amdgpu_buffer_rsrc_t cr = mx_resource(p.w[0] + c0 * row_codes, left * row_codes);
        const __amdgpu_buffer_rsrc_t sr = mx_resource(p.w_scales[0] + c0 * blocks, left * blocks);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            codes[par][i] = __builtin_bit_cast(
                u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                             cr, ((r & 7) + 8 * (i & 1)) * row_codes + 16 * (q + 4 * (r >> 3) + 8 * (i >> 1)), 256 * window,
                             kStreamedOnce));
        scales[par] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(sr, r * blocks, 16 * window, 0));
    };
    const int m = min(r, rows - 1);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    int block = first, window = 0;
    auto next = [&](int& b, int& w) {
        if (++w == windows) {
            w = 0;
            b += stride;
        }
    };
    auto use = [&](int window, auto ic) {
        constexpr int par = decltype(ic)::value;
        // from whole lines to the operands: loads 2 h and 2 h + 1 hold blocks 8 h .. 8 h + 7 of columns
        // 0 .. 7 and 8 .. 15, the operands blocks 8 h .. and 8 h + 4 .. of all sixteen
#pragma unroll
        for (int i = 0; i < 4; i += 2)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t low = codes[par][i][d], high = codes[par][i + 1][d];
                codes[par][i][d] = half_row_move<0xC>(low, high);
                codes[par][i + 1][d] = half_row_move<0x3>(high, low);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = 16 * window + 4 * i + q;               // this lane's block of the row
            const uint32_t e = (scales[par][i] >> (8 * q)) & 0xFFu;
            if constexpr (X == MxX::kBf16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(lds + m * x_pitch + 16 * ((4 * b + j) ^ m));
                    acc = mfma16x16x32(__builtin_bit_cast(bf16x8_t, mx_decode_word(codes[par][i][j], mx_scale(e))),
                                       __builtin_bit_cast(bf16x8_t, x), acc);
                }
            } else {
                const u32x4_t x = *reinterpret_cast<const u32x4_t*>(lds + m * x_pitch + 16 * (b ^ m));
                acc = mx_mfma16(codes[par][i], e, x, xs_scale[m * blocks + b], acc);
            }
        }
    };
    auto finish = [&](int block) {
        const int n = 16 * block + 4 * q;
        if (r < rows && n < p.N) {
            uint16_t* out = p.y[0] + static_cast<size_t>(r) * p.N + n;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) out[e] = f32_to_bf16_bits(acc[e]);
        }
        acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    load(block, window, Even{});
    auto turn = [&](auto ic, auto nc) {
        int b = block, w = window;
        next(b, w);
        load(b, w, nc);
        use(window, ic);
        if (w == 0) finish(block);
        block = b;
        window = w;
    };
    while (block < column_blocks) {
        turn(Even{}, Odd{});
        if (block >= column_blocks) break;
        turn(Odd{}, Even{});
    }
}

}  // namespace

bool mx_qmv_shape(MxOperands op, int sets, int M, int N, int K, int cus, bool whole, MxQmvShape* out) {
    if (M > kMxQmvRows || op == MxOperands::kColumns) return false;
    const bool codes = op == MxOperands::kCodes;
    // The wide form where its waves find work for a few of its latencies.  Measured (K = 2560; narrow /
    // wide us): 8 rows of 8192 columns 7.6 / 9.3, of 12288 10.9 / 9.4, of 32768 22.8 / 11.1; 4 rows of
    // 16384 10.2 / 9.6; one row of 16384 8.7 / 9.5, of 24576 11.6 / 10.3; 16 rows of 16384 with K = 4096
    // (one workgroup per compute unit) 21.3 / 16.5.
    const size_t x_bytes = static_cast<size_t>(M) * (codes ? K / 2 + K / kMxBlock : 2 * K);
    const int column_blocks = (N + 15) / 16;
    out->wide = whole && sets == 1 && K % 512 == 0 && x_bytes <= 160 * 1024 &&
                column_blocks >= (M <= 1 ? 5 : M <= 4 ? 4 : 3) * static_cast<int64_t>(cus);
    if (out->wide) {
        const int resident = std::min<int>(3, static_cast<int>(160 * 1024 / x_bytes));
        out->groups = std::min((column_blocks + kMxWideWaves - 1) / kMxWideWaves, resident * cus);
        out->rows = 16;
        out->columns = 16;
        out->waves = kMxWideWaves;
        out->share = out->batch = 4;
        out->lds = x_bytes;
        return true;
    }
    out->rows = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : M <= 8 ? 8 : 16;
    const int S = out->rows <= 4 ? 4 : 16 / out->rows;
    out->columns = 16 / S;
    out->groups = (N + out->columns - 1) / out->columns;
    const int units = (K / kMxBlock + 4 * S - 1) / (4 * S);
    // Shares of three units (two at 16 rows, whose activations are four loads a unit): one unit a wave
    // leaves more waves than are resident at once.  Measured, one / three units a wave, us: one row of
    // 9728 x 2560 6.0 / 5.3, of 12000 x 2592 7.2 / 6.3, of 1024 x 2560 3.3 / 3.1; 8 rows of 9728 x 2560
    // 9.2 / 7.9; 16 rows one / two / three 9.7 / 9.6 / 10.6.
    auto waves = [&](int share) { return (units + share - 1) / share; };
    out->share = std::max(waves(kMxQmvWaves), std::min(units, out->rows <= 8 ? 3 : 2));
    // Long contractions: larger shares, of one or two whole batches, and with more than one workgroup a
    // compute unit those that put as many waves on each SIMD (five or six waves put two on some): the
    // first with at most four waves or eight, else with at most eight.  2560 columns, share 3 / as
    // chosen, us: 4 rows of 8192 7.7 / 7.0 (share 4), of 9728 8.4 / 8.4, of the gated pair 11.8 / 11.1
    // (6); 8 rows of 8192 10.1 / 8.8 (4), of 9728 11.4 / 10.9, of the gated pair 16.4 / 14.3 (6); 4
    // rows of 14336 on 4096 columns 17.3 / 13.6 (8).  One workgroup a unit wants its loads spread
    // instead (one row of 9728 on 1024 columns 4.2 with shares of 3, 4.4 of 6).  16 rows of 9728, share
    // 5 / 8: 12.9 / 12.0, of 8192 (4 / 8) 10.4 / 10.5.
    if (out->rows <= 8 && out->groups > cus && waves(3) > 4 && waves(3) != 8) {
        int share = 0;
        for (int s : {4, 6, 8})
            if (!share && (waves(s) <= 4 || waves(s) == 8)) share = s;
        for (int s : {4, 6, 8})
            if (!share && waves(s) <= 8) share = s;
        out->share = std::max(waves(kMxQmvWaves), share ? share : 8);
    } else if (out->rows == 16 && units > 64) {
        out->share = std::max(out->share, 8);
    }
    out->waves = waves(out->share);
    const int turns = (out->share + 3) / 4;
    out->batch = (out->share + turns - 1) / turns;
    const size_t x = static_cast<size_t>(out->rows) * S * 256 * out->waves;
    const size_t sums = static_cast<size_t>(sets) * out->waves * S * out->columns * out->columns * sizeof(float);
    out->lds = std::max(x, sums);
    return true;
}

hipError_t launch_mx_qmv(MxOperands op, MxEpilogue epi, bool quantize, const MxTileArgs& args, int cus,
                         hipStream_t stream) {
    MxQmvShape s;
    const int sets = epi == MxEpilogue::kGlu ? 2 : 1;
    const bool whole = (reinterpret_cast<uintptr_t>(args.w_scales[0]) & 15) == 0;
    if (!mx_qmv_shape(op, sets, args.M, args.N, args.L, cus, whole, &s)) return hipErrorInvalidValue;
    const dim3 grid(s.groups), block(64 * s.waves);
    auto run = [&](auto kernel) {
        W4A16_LAUNCH(kernel, grid, block, s.lds, stream, args, s.share);
        return hipGetLastError();
    };
    auto batched = [&](auto cc, auto rc, auto nc) {
        constexpr MxX x = decltype(cc)::value;
        constexpr int rows = decltype(rc)::value, np = decltype(nc)::value;
        if (s.batch == 1) return run(mx_qmv_kernel<x, rows, np, 1>);
        if (s.batch == 2) return run(mx_qmv_kernel<x, rows, np, 2>);
        if (s.batch == 3) return run(mx_qmv_kernel<x, rows, np, 3>);
        return run(mx_qmv_kernel<x, rows, np, 4>);
    };
    auto sized = [&](auto cc, auto nc) {
        if constexpr (decltype(cc)::value != MxX::kCodes) {
            if (s.rows == 1) return batched(cc, std::integral_constant<int, 1>{}, nc);
            if (s.rows == 2) return batched(cc, std::integral_constant<int, 2>{}, nc);
        }
        if (s.rows <= 4) return batched(cc, std::integral_constant<int, 4>{}, nc);
        if (s.rows == 8) return batched(cc, std::integral_constant<int, 8>{}, nc);
        return batched(cc, std::integral_constant<int, 16>{}, nc);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Bf16 = std::integral_constant<MxX, MxX::kBf16>;
    using Codes = std::integral_constant<MxX, MxX::kCodes>;
    using Quantize = std::integral_constant<MxX, MxX::kQuantize>;
    if (s.wide) {
        auto wide = [&](auto kernel) {
            W4A16_LAUNCH(kernel, dim3(s.groups), dim3(64 * kMxWideWaves), s.lds, stream, args);
            return hipGetLastError();
        };
        if (op == MxOperands::kRows) return wide(mx_qmv_wide_kernel<MxX::kBf16>);
        return quantize ? wide(mx_qmv_wide_kernel<MxX::kQuantize>) : wide(mx_qmv_wide_kernel<MxX::kCodes>);
    }
    if (op == MxOperands::kCodes) return quantize ? sized(Quantize{}, One{}) : sized(Codes{}, One{});
    return sets == 2 ? sized(Bf16{}, Two{}) : sized(Bf16{}, One{});
}

}  // namespace w4a16
