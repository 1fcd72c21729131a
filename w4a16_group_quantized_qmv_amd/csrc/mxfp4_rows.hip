// Quantization of rows to MXFP4 and back.
//
//   a = max |x| of a block;  e = max(floor(log2 a) - 2, -127) + 127  (a = 0 gives e = 0);
//   code = x / 2^(e - 127) rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, a tie to the code
//   with an even mantissa bit, and values above 6 (at most 8 by the choice of e) to 6; the sign of x.
// A block with an infinity or a NaN gets e = 255 (NaN) and codes 0, so that it cannot pass for
// numbers.  Both directions are exact otherwise: scaling by a power of two rounds nothing that the
// grid keeps, and what a block of finite values is encoded to (e <= 252) is a bf16 value.  Bytes 253 and
// 254 from elsewhere can stand for 2^128 and more, past bf16: those values become infinities.
//
// Bound by memory: 2 (or 4) bytes read and 0.53 written per value.  Rows are contiguous and a whole
// number of blocks, so the array is a flat list of blocks.  Four lanes share a block, eight values
// each: every load is 16 bytes per lane over consecutive addresses, the maximum takes two
// lane exchanges, and a wave's codes are 256 consecutive bytes.
// Measured on MI355X: 4096 x 9728 bf16 17.3 us (5.8 TB/s), 9728 x 2560 fp32 16.5 us (6.8, the
// input in the last-level cache from the call before); 33 x 2560 2.3 us, a launch and two memory latencies.
#include "mxfp4_device.h"
#include "mxfp4_internal.h"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kRowThreads = 256;

// fp32 bits of |v|: comparing them as integers orders finite values, infinities and NaN alike.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The value of another lane of the same four (DPP quad_perm).
template <int PERM>
__device__ __forceinline__ uint32_t quad_exchange(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), PERM, 0xF, 0xF, true));
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void mx_quantize_kernel(const void* __restrict__ x,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales, int64_t chunks) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; c < chunks; c += stride) {
        float v[8];
        if constexpr (F32) {
            const u32x4_t lo = load16(static_cast<const float*>(x) + 8 * c);
            const u32x4_t hi = load16(static_cast<const float*>(x) + 8 * c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(lo[i]);
                v[4 + i] = __uint_as_float(hi[i]);
            }
        } else {
            const u32x4_t w = load16(static_cast<const uint16_t*>(x) + 8 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
        // chunks is a multiple of four, so the four lanes of a block are in the loop together
        top = max(top, quad_exchange<0xB1>(top));    // lanes 1 0 3 2
        top = max(top, quad_exchange<0x4E>(top));    // lanes 2 3 0 1
        // The exponent field less 2.  It is 0 for fp32 subnormals, which lie below 2^-126: their
        // e is 0 as well (2^-127 is the smallest scale).
        const uint32_t field = top >> 23;
        const uint32_t e = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
        const float scale = mx_scale(e);
        uint32_t word = 0;
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[0], v[1], scale, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[2], v[3], scale, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[4], v[5], scale, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[6], v[7], scale, 3);
        codes[c] = e == 255u ? 0u : word;
        if ((c & 3) == 0) scales[c >> 2] = static_cast<uint8_t>(e);
    }
}

__global__ __launch_bounds__(kRowThreads) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ scales,
                                                                    u32x4_t* __restrict__ y, int64_t chunks) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; c < chunks; c += stride)
        y[c] = mx_decode_word(codes[c], mx_scale(scales[c >> 2]));
}

// Eight values of a padded row per thread.
__global__ __launch_bounds__(kRowThreads) void mx_pad_rows_kernel(const uint16_t* __restrict__ x, u32x4_t* __restrict__ y,
                                                                  int64_t chunks, int N) {
    const int per_row = (N + 7) / 8;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; c < chunks; c += stride) {
        const int64_t row = c / per_row;
        const int n = static_cast<int>(c - row * per_row) * 8;
        const uint16_t* in = x + row * N + n;
        u32x4_t v = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N) v[i >> 1] |= static_cast<uint32_t>(in[i]) << (16 * (i & 1));
        y[c] = v;
    }
}

// Sums of split-K partials, in slice order: y = bf16(sum_z ws[z]) or, for the gated pair,
// silu(sum_z ws[0][z]) * sum_z ws[1][z].  Four outputs per thread; the loads of up to eight slices are
// issued before the first sum, since a load that waits for the one before it costs a memory latency
// per slice (eight slices of 64 x 2560 outputs: 7.7 us that way).
template <int SETS, int S>
__global__ __launch_bounds__(kRowThreads) void mx_sum_kernel(const float* __restrict__ ws, uint16_t* __restrict__ y,
                                                             int64_t MN, int split) {
    const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x);
    if (i >= MN) return;
    const bool whole = MN % 4 == 0;          // every slice starts on 16 bytes
    f32x4_t v[SETS];
#pragma unroll
    for (int s = 0; s < SETS; ++s) v[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int z0 = 0; z0 < split; z0 += S) {
        f32x4_t part[SETS][S];
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int z = 0; z < S; ++z) {
                const float* in = ws + (static_cast<int64_t>(s) * split + min(z0 + z, split - 1)) * MN + i;
                if (whole) {
                    part[s][z] = *reinterpret_cast<const f32x4_t*>(in);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) part[s][z][e] = i + e < MN ? in[e] : 0.f;
                }
            }
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int z = 0; z < S; ++z)
                if (z0 + z < split) v[s] += part[s][z];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float r = v[0][e];
        if constexpr (SETS == 2) r = r * mx_sigmoid(r) * v[SETS - 1][e];
        if (i + e < MN) y[i + e] = f32_to_bf16_bits(r);
    }
}

// Workgroups: one pass over small arrays; above that 8192 (32 for each of 256 compute units, four
// times what is resident at once), which take chunk after chunk.
int row_grid(int64_t chunks) {
    return static_cast<int>(std::min<int64_t>((chunks + kRowThreads - 1) / kRowThreads, 256 * 32));
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, bool x_fp32, uint8_t* codes, uint8_t* scales, int64_t blocks,
                              hipStream_t stream) {
    const int64_t chunks = 4 * blocks;
    uint32_t* words = reinterpret_cast<uint32_t*>(codes);
    if (x_fp32)
        hipLaunchKernelGGL(mx_quantize_kernel<true>, dim3(row_grid(chunks)), dim3(kRowThreads), 0, stream, x, words,
                           scales, chunks);
    else
        hipLaunchKernelGGL(mx_quantize_kernel<false>, dim3(row_grid(chunks)), dim3(kRowThreads), 0, stream, x, words,
                           scales, chunks);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, uint16_t* y, int64_t blocks,
                                hipStream_t stream) {
    const int64_t chunks = 4 * blocks;
    hipLaunchKernelGGL(mx_dequantize_kernel, dim3(row_grid(chunks)), dim3(kRowThreads), 0, stream,
                       reinterpret_cast<const uint32_t*>(codes), scales, reinterpret_cast<u32x4_t*>(y), chunks);
    return hipGetLastError();
}

hipError_t launch_mx_pad_rows(const uint16_t* x, uint16_t* y, int64_t M, int N, hipStream_t stream) {
    const int64_t chunks = M * ((N + 7) / 8);
    hipLaunchKernelGGL(mx_pad_rows_kernel, dim3(row_grid(chunks)), dim3(kRowThreads), 0, stream, x,
                       reinterpret_cast<u32x4_t*>(y), chunks, N);
    return hipGetLastError();
}

hipError_t launch_mx_sum(const float* ws, uint16_t* y, int sets, int64_t MN, int split, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>((MN + 4 * kRowThreads - 1) / (4 * kRowThreads))), block(kRowThreads);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, ws, y, MN, split);
        return hipGetLastError();
    };
    if (sets == 2) return split <= 2 ? run(mx_sum_kernel<2, 2>) : split <= 4 ? run(mx_sum_kernel<2, 4>) : run(mx_sum_kernel<2, 8>);
    return split <= 2 ? run(mx_sum_kernel<1, 2>) : split <= 4 ? run(mx_sum_kernel<1, 4>) : run(mx_sum_kernel<1, 8>);
}

}  // namespace w4a16
