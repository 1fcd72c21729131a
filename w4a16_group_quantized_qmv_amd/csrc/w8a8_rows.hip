// Rows of int8 codes: the quantizer, and the sum of a split product's slices.
#include "w8a8_device.h"
#include "w8a8_internal.h"

namespace w4a16 {
namespace {

// A workgroup of WAVES waves per row.  The row's magnitudes are reduced first, its codes made from a second
// read, which comes from the L2 (a row is at most 512 KB).
template <bool FP32, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w8_quantize_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales, int K) {
    constexpr int NT = 64 * WAVES;
    __shared__ float red[WAVES];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, chunks = K / 8;
    const uint8_t* in = static_cast<const uint8_t*>(x) + row * K * (FP32 ? 4 : 2);
    auto load8 = [&](int c, float (&v)[8]) {
        if constexpr (FP32) {
            const u32x4_t a = load16(in + 32 * static_cast<size_t>(c)), b = load16(in + 32 * static_cast<size_t>(c) + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(b[i]);
            }
        } else {
            const u32x4_t a = load16(in + 16 * static_cast<size_t>(c));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
            }
        }
    };
    // magnitudes as integers keep their order, and a NaN comes out above an infinity
    uint32_t top = 0;
    for (int c = tid; c < chunks; c += NT) {
        float v[8];
        load8(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, 64)));
    if constexpr (WAVES > 1) {
        if ((tid & 63) == 0) red[tid >> 6] = __uint_as_float(top);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = max(top, __float_as_uint(red[i]));
    }
    float inverse, scale;
    w8_row_scale(__uint_as_float(top), inverse, scale);
    if (tid == 0) scales[row] = scale;
    for (int c = tid; c < chunks; c += NT) {
        float v[8];
        load8(c, v);
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo |= w8_code(v[i], inverse) << (8 * i);
            hi |= w8_code(v[4 + i], inverse) << (8 * i);
        }
        *reinterpret_cast<uint2*>(codes + row * K + 8 * static_cast<int64_t>(c)) = make_uint2(lo, hi);
    }
}

// Slices are int32, so their sum is exact in any order.
__global__ __launch_bounds__(256) void w8_sum_kernel(const int* __restrict__ ws, const float* __restrict__ a_scales,
                                                     const float* __restrict__ w_scales, uint16_t* __restrict__ y,
                                                     int64_t M, int N, int split) {
    const int64_t MN = M * N, at = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
    if (at >= MN) return;
    const int count = static_cast<int>(min(static_cast<int64_t>(4), MN - at));
    int sum[4] = {0, 0, 0, 0};
    const bool wide = count == 4 && MN % 4 == 0;
    for (int s = 0; s < split; ++s) {
        const int* in = ws + s * MN + at;
        if (wide) {
            const i32x4_t v = *reinterpret_cast<const i32x4_t*>(in);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < count) sum[e] += in[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (e >= count) break;
        const int64_t m = (at + e) / N;
        const int n = static_cast<int>((at + e) - m * N);
        y[at + e] = f32_to_bf16_bits(static_cast<float>(sum[e]) * w_scales[n] * a_scales[m]);
    }
}

}  // namespace

hipError_t launch_w8_quantize(const void* x, bool x_fp32, int8_t* codes, float* scales, int64_t R, int K,
                              hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(R));
    if (x_fp32)
        hipLaunchKernelGGL((w8_quantize_kernel<true, 4>), grid, dim3(256), 0, stream, x, codes, scales, K);
    else
        hipLaunchKernelGGL((w8_quantize_kernel<false, 4>), grid, dim3(256), 0, stream, x, codes, scales, K);
    return hipGetLastError();
}

hipError_t launch_w8_sum(const int* ws, const float* a_scales, const float* w_scales, uint16_t* y, int64_t M, int N,
                         int split, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>((M * N + 1023) / 1024));
    hipLaunchKernelGGL(w8_sum_kernel, grid, dim3(256), 0, stream, ws, a_scales, w_scales, y, M, N, split);
    return hipGetLastError();
}

}  // namespace w4a16
