// Products of int8 weights for decode rows: at most 16 rows of one matrix, or few rows of each of many experts.
//
//   y[m, n] = x_scale[m] w_scale[n] sum_k a[m, k] w[n, k]      h[m, n] = silu(g[m, n]) u[m, n]
//
// Bound by memory: every weight is read once (one byte) and used by a few rows, so all of a matrix has to be
// asked for within about one memory latency.
//  * A workgroup has 16 weight rows (of each set); its waves take consecutive shares of the contraction.  A unit
//    is 1 KB: 64 codes of each of the 16 rows, 16 bytes a lane, one 16x16x64 MFMA.  A wave issues the loads of a
//    batch of units before it uses the first.
//  * The activations come as codes, or as bf16 and are quantized by every workgroup for itself, while its first
//    weights are on their way: a launch less, for reading the rows again in each workgroup (from L2).
//  * The waves' int32 sums are added by the first wave; integers, so in any order.
#include "w8a8_device.h"
#include "w8a8_internal.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

template <int NP, bool EXPERTS, bool QUANTIZE, int UB>
__global__ __launch_bounds__(64 * kW8QmvWaves) void w8_qmv_kernel(const W8TileArgs p, int rows_max, int share,
                                                                  int column_blocks) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int K = p.K, N = p.N, chunks = K / kW8Chunk, units = (chunks + 3) / 4;

    int expert = 0, m0 = 0, rows = p.R, cb;
    if constexpr (EXPERTS) {
        ExpertTile tile;
        if (!find_expert_tile<1>(p.offsets, p.E, p.R, rows_max, column_blocks, blockIdx.x, tile)) return;
        expert = tile.expert;
        m0 = tile.first + tile.tm * rows_max;
        rows = min(tile.end - m0, rows_max);
        cb = tile.tn;
    } else {
        cb = xcd_remap(blockIdx.x, column_blocks);
    }
    const int c0 = cb * kW8QmvColumns;
    auto source_row = [&](int r) {       // the activation row of row r of this workgroup; -1 for none
        if (r >= rows) return -1;
        if (!EXPERTS || p.tokens == nullptr) return m0 + r;
        const int t = p.tokens[m0 + r];
        return t >= 0 && t < p.T ? t : -1;
    };

    // ---- weights: lane l has codes 16 (l / 16) .. of row l % 16 of a unit
    const int64_t w_base = (static_cast<int64_t>(expert) * N + c0) * K, w_bytes = static_cast<int64_t>(N - c0) * K;
    const __amdgpu_buffer_rsrc_t wr0 = mx_resource(p.w[0] + w_base, w_bytes);
    const __amdgpu_buffer_rsrc_t wr1 = NP > 1 ? mx_resource(p.w[1] + w_base, w_bytes) : wr0;
    const uint32_t w_off = static_cast<uint32_t>(lane & 15) * static_cast<uint32_t>(K) + 16u * (lane >> 4);
    const int u_begin = wave * share, u_end = min(u_begin + share, units);
    u32x4_t w[NP][UB];
    auto load_batch = [&](int u0) {
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int u = u0 + i;
            const uint32_t o = u < u_end && 4 * u + (lane >> 4) < chunks ? w_off : kOutside;
#pragma unroll
            for (int s = 0; s < NP; ++s)
                w[s][i] = __builtin_bit_cast(
                    u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(s ? wr1 : wr0, o, 64 * u, kStreamedOnce));
        }
    };
    load_batch(u_begin);

    // ---- activations: row r at r * (K + 16) in LDS, its scale behind the rows and the waves' sums
    const int pitch = K + 16;
    float* row_scale = reinterpret_cast<float*>(lds);                                  // [16]
    uint32_t* tops = reinterpret_cast<uint32_t*>(lds + 64);                            // [16][waves]
    i32x4_t* sums = reinterpret_cast<i32x4_t*>(lds + 64 + 64 * kW8QmvWaves);           // [NP][waves][64]
    uint8_t* codes = lds + 64 + 64 * kW8QmvWaves + NP * waves * 1024;
    if constexpr (QUANTIZE) {
        const int pieces = K / 8, threads = blockDim.x;
        for (int r = 0; r < rows; ++r) {
            const int m = source_row(r);
            uint32_t top = 0;
            if (m >= 0)
                for (int c = tid; c < pieces; c += threads) {
                    const u32x4_t v = load16(p.x + static_cast<int64_t>(m) * K + 8 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = max(top, max((v[i] << 16) & 0x7FFF0000u, v[i] & 0x7FFF0000u));
                }
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, 64)));
            if (lane == 0) tops[r * kW8QmvWaves + wave] = top;
        }
        __syncthreads();
        for (int r = 0; r < rows; ++r) {
            const int m = source_row(r);
            uint32_t top = 0;
            for (int i = 0; i < waves; ++i) top = max(top, tops[r * kW8QmvWaves + i]);
            float inverse, scale;
            w8_row_scale(__uint_as_float(top), inverse, scale);
            if (tid == 0) row_scale[r] = scale;
            for (int c = tid; c < pieces; c += threads) {
                uint32_t lo = 0, hi = 0;
                if (m >= 0) {
                    const u32x4_t v = load16(p.x + static_cast<int64_t>(m) * K + 8 * c);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        lo |= w8_code(__uint_as_float(v[i] << 16), inverse) << (16 * i);
                        lo |= w8_code(__uint_as_float(v[i] & 0xFFFF0000u), inverse) << (16 * i + 8);
                        hi |= w8_code(__uint_as_float(v[2 + i] << 16), inverse) << (16 * i);
                        hi |= w8_code(__uint_as_float(v[2 + i] & 0xFFFF0000u), inverse) << (16 * i + 8);
                    }
                }
                *reinterpret_cast<uint2*>(codes + r * pitch + 8 * c) = make_uint2(lo, hi);
            }
        }
        __syncthreads();
    }
    // lanes of rows that are none read a zero operand
    const int own_row = QUANTIZE ? ((lane & 15) < rows ? lane & 15 : -1) : source_row(lane & 15);
    const int8_t* global_row = p.a + static_cast<int64_t>(max(own_row, 0)) * K;
    auto activation = [&](int u) {
        const int c = 4 * u + (lane >> 4);
        if (own_row < 0 || u >= u_end || c >= chunks) return u32x4_t{0, 0, 0, 0};
        if constexpr (QUANTIZE) return *reinterpret_cast<const u32x4_t*>(codes + own_row * pitch + 16 * c);
        else return load16(global_row + 16 * c);
    };

    i32x4_t acc[NP];
#pragma unroll
    for (int s = 0; s < NP; ++s) acc[s] = i32x4_t{0, 0, 0, 0};
    for (int u0 = u_begin; u0 < u_end; u0 += UB) {
        if (u0 > u_begin) load_batch(u0);
        u32x4_t a[UB];
#pragma unroll
        for (int i = 0; i < UB; ++i) a[i] = activation(u0 + i);
#pragma unroll
        for (int i = 0; i < UB; ++i)
#pragma unroll
            for (int s = 0; s < NP; ++s) acc[s] = mfma16_i8(w[s][i], a[i], acc[s]);
    }
#pragma unroll
    for (int s = 0; s < NP; ++s) sums[(s * waves + wave) * 64 + lane] = acc[s];
    __syncthreads();
    if (wave != 0) return;

    // Lane l has columns 4 (l / 16) .. + 3 of row l % 16.
    float v[NP][4];
    const int r = lane & 15, n = c0 + 4 * (lane >> 4);
    const int m = source_row(r);
    const float xs = m < 0 ? 0.f : QUANTIZE ? row_scale[r] : p.a_scales[m];
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        i32x4_t sum = {0, 0, 0, 0};
        for (int i = 0; i < waves; ++i) sum += sums[(s * waves + i) * 64 + lane];
        const float* scales = p.w_scales[s] + static_cast<int64_t>(expert) * N;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[s][e] = static_cast<float>(sum[e]) * (n + e < N ? scales[n + e] : 0.f) * xs;
    }
    if (r >= rows) return;
    uint16_t* out = p.y[0] + static_cast<int64_t>(m0 + r) * N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float y = NP == 1 ? v[0][e] : v[0][e] * mx_sigmoid(v[0][e]) * v[NP - 1][e];
        if (n + e < N) out[e] = f32_to_bf16_bits(y);
    }
}

}  // namespace

// At most 64 KB of activations, so that a second workgroup fits beside.
bool w8_qmv_shape(int sets, int rows, int K, bool quantize, W8QmvShape* out) {
    const int units = (K + 63) / 64;
    out->rows = rows;
    out->waves = std::max(1, std::min(kW8QmvWaves, (units + 3) / 4));
    out->share = (units + out->waves - 1) / out->waves;
    out->batch = out->share <= 4 || sets > 1 ? 4 : 8;
    const size_t codes = quantize ? static_cast<size_t>(rows) * (K + 16) : 0;
    out->lds = 64 + 64 * kW8QmvWaves + static_cast<size_t>(sets) * out->waves * 1024 + codes;
    return codes <= 65536;
}

namespace {

template <int NP, bool EXPERTS>
hipError_t launch_form(const W8TileArgs& args, const W8QmvShape& s, hipStream_t stream) {
    const int blocks = (args.N + kW8QmvColumns - 1) / kW8QmvColumns;
    const int pieces = EXPERTS ? static_cast<int>(std::min<int64_t>(args.R, args.R / s.rows + args.E)) : 1;
    const dim3 grid(static_cast<uint32_t>(pieces) * blocks), block(64 * s.waves);
    auto run = [&](auto kernel) {
        if (s.lds > 65536) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(s.lds));
            if (e != hipSuccess) return e;
        }
        W4A16_LAUNCH(kernel, grid, block, s.lds, stream, args, s.rows, s.share, blocks);
        return hipGetLastError();
    };
    auto batch = [&](auto qc) {
        constexpr bool q = decltype(qc)::value;
        return s.batch <= 4 ? run(w8_qmv_kernel<NP, EXPERTS, q, 4>) : run(w8_qmv_kernel<NP, EXPERTS, q, 8>);
    };
    return args.x ? batch(std::true_type{}) : batch(std::false_type{});
}

}  // namespace

hipError_t launch_w8_qmv(W8Epilogue epi, int rows, const W8TileArgs& args, hipStream_t stream) {
    W8QmvShape s;
    const int sets = epi == W8Epilogue::kStore ? 1 : 2;
    if (epi == W8Epilogue::kGluGrad || !w8_qmv_shape(sets, rows, args.K, args.x != nullptr, &s)) return hipErrorInvalidValue;
    if (!args.offsets) return sets == 1 ? launch_form<1, false>(args, s, stream) : hipErrorInvalidValue;
    return sets == 1 ? launch_form<1, true>(args, s, stream) : launch_form<2, true>(args, s, stream);
}

}  // namespace w4a16
