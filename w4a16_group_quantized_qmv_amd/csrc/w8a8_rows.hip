// Rows of int8 codes: the quantizer, and the sum of a split product's slices.
#include "w8a8_device.h"
#include "w8a8_internal.h"

#include <type_traits>

namespace w4a16 {
namespace {

// WAVES waves per row, HELD chunks of eight values a lane: they stay in registers between the reduction of the row's
// magnitudes and its codes (HELD 0: longer rows are read twice, the second time from the L2).  Bound by reading
// and writing once: 4096 x 2560 bf16, 31 MB, takes 8.6 us, 3.7 TB/s, and 6.4 us the same rows again; fp32, 52 MB, 9.3 us
// (4096 x 9728: 20.0 and 30.1 us).
template <bool FP32, int WAVES, int HELD>
__global__ __launch_bounds__(256) void w8_quantize_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int64_t R, int K) {
    constexpr int NT = 64 * WAVES, ROWS = 4 / WAVES;
    __shared__ uint32_t red[4];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / NT;
    const int tid = threadIdx.x % NT, chunks = K / 8;
    if (WAVES < 4 && row >= R) return;
    const uint8_t* in = static_cast<const uint8_t*>(x) + row * K * (FP32 ? 4 : 2);
    struct Chunk {
        u32x4_t a, b;
    };
    auto load = [&](int c) {
        Chunk v{};
        if constexpr (FP32) {
            v.a = load16(in + 32 * static_cast<size_t>(c));
            v.b = load16(in + 32 * static_cast<size_t>(c) + 16);
        } else {
            v.a = load16(in + 16 * static_cast<size_t>(c));
        }
        return v;
    };
    auto value = [](const Chunk& v, int i) {
        if constexpr (FP32) return __uint_as_float(i < 4 ? v.a[i] : v.b[i - 4]);
        else return __uint_as_float((i & 1) ? v.a[i / 2] & 0xFFFF0000u : v.a[i / 2] << 16);
    };
    // magnitudes as integers keep their order, and a NaN comes out above an infinity
    uint32_t top = 0;
    auto reduce = [&](const Chunk& v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(value(v, i)) & 0x7FFFFFFFu);
    };
    Chunk held[HELD > 0 ? HELD : 1];
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i] = tid + i * NT < chunks ? load(tid + i * NT) : Chunk{};
#pragma unroll
        for (int i = 0; i < HELD; ++i) reduce(held[i]);
    } else {
        for (int c = tid; c < chunks; c += NT) reduce(load(c));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, 64)));
    if constexpr (WAVES > 1) {
        if ((tid & 63) == 0) red[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = max(top, red[i]);
    }
    float inverse, scale;
    w8_row_scale(__uint_as_float(top), inverse, scale);
    if (tid == 0) scales[row] = scale;
    auto store = [&](int c, const Chunk& v) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo |= w8_code(value(v, i), inverse) << (8 * i);
            hi |= w8_code(value(v, 4 + i), inverse) << (8 * i);
        }
        *reinterpret_cast<uint2*>(codes + row * K + 8 * static_cast<int64_t>(c)) = make_uint2(lo, hi);
    };
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (tid + i * NT < chunks) store(tid + i * NT, held[i]);
    } else {
        for (int c = tid; c < chunks; c += NT) store(c, load(c));
    }
}

// Four columns a thread, S slices on their way at a time.  Slices are int32, so their sum is exact in any order.  WIDE:
// columns in whole fours, in rows of their own.  Bound by latency and by reading them (three of 509 x 2560, 18 MB: 4.2 us;
// slice after slice, with a division for each value, 5.3).
template <int S, bool WIDE>
__global__ __launch_bounds__(256) void w8_sum_kernel(const int* __restrict__ ws, const float* __restrict__ a_scales,
                                                     const float* __restrict__ w_scales, uint16_t* __restrict__ y,
                                                     int64_t M, int N, int split) {
    const uint32_t four = blockIdx.x * 256u + threadIdx.x;      // (below 2^32, as the call checks)
    const int64_t MN = M * N, at = 4 * static_cast<int64_t>(four);
    if (at >= MN) return;
    i32x4_t sum = {0, 0, 0, 0};
    for (int z0 = 0; z0 < split; z0 += S) {
        i32x4_t part[S];
#pragma unroll
        for (int z = 0; z < S; ++z) {
            const int* in = ws + min(z0 + z, split - 1) * MN + at;
            if constexpr (WIDE) {
                part[z] = *reinterpret_cast<const i32x4_t*>(in);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) part[z][e] = at + e < MN ? in[e] : 0;
            }
        }
#pragma unroll
        for (int z = 0; z < S; ++z)
            if (z0 + z < split) sum += part[z];
    }
    if constexpr (WIDE) {
        const uint32_t row_fours = static_cast<uint32_t>(N) / 4, m = four / row_fours, n = 4 * (four - m * row_fours);
        const float xs = a_scales[m];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(sum[e]) * w_scales[n + e] * xs;
        *reinterpret_cast<uint2*>(y + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (at + e >= MN) break;
            const int64_t m = (at + e) / N;
            y[at + e] = f32_to_bf16_bits(static_cast<float>(sum[e]) * w_scales[(at + e) - m * N] * a_scales[m]);
        }
    }
}

}  // namespace

hipError_t launch_w8_quantize(const void* x, bool x_fp32, int8_t* codes, float* scales, int64_t R, int K,
                              hipStream_t stream) {
    // a wave per row up to 4096 values, a workgroup beyond; 2^23 rows a launch, whose threads stay below 2^32
    constexpr int64_t kRows = int64_t{1} << 23;
    if (R > kRows) {
        for (int64_t r = 0; r < R; r += kRows) {
            const hipError_t e = launch_w8_quantize(static_cast<const uint8_t*>(x) + r * K * (x_fp32 ? 4 : 2), x_fp32, codes + r * K,
                                                    scales + r, R - r < kRows ? R - r : kRows, K, stream);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    auto form = [&](auto tc) {
        constexpr bool FP32 = decltype(tc)::value;
        auto run = [&](auto kernel, int rows) {
            hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>((R + rows - 1) / rows)), dim3(256), 0, stream, x, codes, scales, R, K);
            return hipGetLastError();
        };
        if (K <= 1024) return run(w8_quantize_kernel<FP32, 1, 2>, 4);
        if (K <= 2560) return run(w8_quantize_kernel<FP32, 1, 5>, 4);
        if (K <= 4096) return run(w8_quantize_kernel<FP32, 1, 8>, 4);
        if (K <= 10240) return run(w8_quantize_kernel<FP32, 4, 5>, 1);
        return run(w8_quantize_kernel<FP32, 4, 0>, 1);
    };
    return x_fp32 ? form(std::true_type{}) : form(std::false_type{});
}

hipError_t launch_w8_sum(const int* ws, const float* a_scales, const float* w_scales, uint16_t* y, int64_t M, int N,
                         int split, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>((M * N + 1023) / 1024));
    const bool wide = N % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, ws, a_scales, w_scales, y, M, N, split);
        return hipGetLastError();
    };
    if (!wide) return run(w8_sum_kernel<4, false>);
    return split <= 2 ? run(w8_sum_kernel<2, true>) : split <= 4 ? run(w8_sum_kernel<4, true>) : run(w8_sum_kernel<8, true>);
}

}  // namespace w4a16
