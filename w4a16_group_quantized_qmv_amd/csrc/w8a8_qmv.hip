// Products of int8 weights for decode rows: at most 16 rows of one matrix.
//
//   y[m, n] = x_scale[m] w_scale[n] sum_k a[m, k] w[n, k]
//
// Bound by memory: every weight is read once (one byte) and used by a few rows, so all of a matrix has to be
// asked for within about one memory latency.
//  * A workgroup has 16 weight rows; its waves take consecutive shares of the contraction.  A wave moves its share
//    to LDS of its own, eight rows by one line of 128 bytes an instruction, up to five lines of every row at once,
//    and waits only for itself.  (Loads to registers in the operand's layout, 64 bytes of 16 rows, took 9.2 us for
//    one row of 9728 x 2560 where this takes 6.4 us: 3.9 TB/s, a launch included.)
//  * 16-byte chunk c of row r lies at c ^ ((r / 2) % 8), as in the tiles.  The 16x16x64 MFMA takes the weight rows
//    as its rows and the activation rows as its columns.
//  * The activations come as codes, or as bf16 and are quantized by every workgroup for itself: a launch less, for
//    reading the rows again in each workgroup (from L2).  They are asked for before the weights, since loads
//    arrive in order.
//  * The waves' int32 sums are added by the first wave; integers, so in any order.
#include "w8a8_device.h"
#include "w8a8_internal.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

constexpr int kLines = 5;       // 128-byte lines of a weight row in flight in a wave
constexpr int kPieces = 4;      // 16-byte pieces of an activation row that a thread quantizes

__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// QROWS: rows that are quantized on the way, 0: codes.  share: lines of a wave.
template <int QROWS>
__global__ __launch_bounds__(64 * kW8QmvWaves) void w8_qmv_kernel(const W8TileArgs p, int share, int column_blocks) {
    constexpr int C = kW8QmvColumns;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int K = p.K, N = p.N, rows = p.R, chunks = K / kW8Chunk, lines = (chunks + 7) / 8;
    const int c0 = xcd_remap(blockIdx.x, column_blocks) * C;

    // LDS: row scales, the waves' largest magnitudes, the rows' codes, and the waves' lines
    float* row_scale = reinterpret_cast<float*>(lds);
    uint32_t* tops = reinterpret_cast<uint32_t*>(lds + 64);
    uint8_t* codes = lds + 64 + 64 * kW8QmvWaves;
    const int pitch = K + 16;
    const int wave_bytes = min(share, kLines) * C * 128;
    uint8_t* own = codes + QROWS * pitch + wave * wave_bytes;

    // ---- weights
    const int l_begin = wave * share, l_end = min(l_begin + share, lines);
    const __amdgpu_buffer_rsrc_t wr = mx_resource(p.w[0] + static_cast<int64_t>(c0) * K, static_cast<int64_t>(N - c0) * K);
    auto load_lines = [&](int l0) {
#pragma unroll
        for (int i = 0; i < kLines; ++i) {
            const int l = l0 + i;
            if (l >= l_end) break;                           // (uniform)
#pragma unroll
            for (int q = 0; q < C / 8; ++q) {
                const int r = 8 * q + (lane >> 3), c = 8 * l + ((lane & 7) ^ ((r >> 1) & 7));
                const uint32_t o = c < chunks ? static_cast<uint32_t>(r) * static_cast<uint32_t>(K) + 16u * c : kOutside;
                uint8_t* to = own + (i * C + 8 * q) * 128;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, to, 16, o, 0, 0, kStreamedOnce);
            }
        }
    };

    // ---- activations: lanes of rows that are none take zeros
    const int own_row = (lane & 15) < rows ? lane & 15 : -1;
    u32x4_t a[2 * kLines];
    auto load_codes = [&](int l0) {
        const int8_t* row = p.a + static_cast<int64_t>(max(own_row, 0)) * K;
#pragma unroll
        for (int i = 0; i < 2 * kLines; ++i) {
            const int c = 8 * l0 + 4 * i + (lane >> 4);
            a[i] = own_row >= 0 && c < min(chunks, 8 * l_end) ? load16(row + 16 * c) : u32x4_t{0, 0, 0, 0};
        }
    };
    if constexpr (QROWS > 0) {
        const int pieces = K / 8, threads = blockDim.x;
        u32x4_t v[QROWS][kPieces];
#pragma unroll
        for (int r = 0; r < QROWS; ++r) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int c = tid + i * threads;
                v[r][i] = r < rows && c < pieces ? load16(p.x + static_cast<int64_t>(r) * K + 8 * c) : u32x4_t{0, 0, 0, 0};
            }
        }
        asm volatile("" ::: "memory");
        load_lines(l_begin);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int r = 0; r < QROWS; ++r) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max((v[r][i][e] << 16) & 0x7FFF0000u, v[r][i][e] & 0x7FFF0000u));
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, 64)));
            if (lane == 0) tops[r * kW8QmvWaves + wave] = top;
        }
        lds_barrier();
#pragma unroll
        for (int r = 0; r < QROWS; ++r) {
            uint32_t top = 0;
            for (int i = 0; i < waves; ++i) top = max(top, tops[r * kW8QmvWaves + i]);
            float inverse, scale;
            w8_row_scale(__uint_as_float(top), inverse, scale);
            if (tid == 0) row_scale[r] = scale;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int c = tid + i * threads;
                if (c >= pieces) continue;
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e >> 1] |= w8_code(__uint_as_float(v[r][i][e] << 16), inverse) << (16 * (e & 1));
                    w[e >> 1] |= w8_code(__uint_as_float(v[r][i][e] & 0xFFFF0000u), inverse) << (16 * (e & 1) + 8);
                }
                *reinterpret_cast<uint2*>(codes + r * pitch + 8 * c) = make_uint2(w[0], w[1]);
            }
        }
        lds_barrier();
    } else {
        load_codes(l_begin);
        asm volatile("" ::: "memory");
        load_lines(l_begin);
    }

    i32x4_t acc = {0, 0, 0, 0};
    const int key = ((lane & 15) >> 1) & 7;
    for (int l0 = l_begin; l0 < l_end; l0 += kLines) {
        if (l0 > l_begin) {
            // (this wave's reads of the lines before are done)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if constexpr (QROWS == 0) load_codes(l0);
            load_lines(l0);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < kLines; ++i) {
            if (l0 + i >= l_end) break;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u32x4_t x;
                const int c = 8 * (l0 + i) + 4 * j + (lane >> 4);
                if constexpr (QROWS > 0)
                    x = own_row >= 0 && c < chunks ? *reinterpret_cast<const u32x4_t*>(codes + own_row * pitch + 16 * c)
                                                   : u32x4_t{0, 0, 0, 0};
                else
                    x = a[2 * i + j];
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(own + (i * C + (lane & 15)) * 128 +
                                                                    16 * ((4 * j + (lane >> 4)) ^ key));
                acc = mfma16_i8(w, x, acc);
            }
        }
    }
    // the sums go where this wave's lines were
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    *reinterpret_cast<i32x4_t*>(own + lane * 16) = acc;
    lds_barrier();
    if (wave != 0) return;

    // Lane l has columns 4 (l / 16) .. + 3 of row l % 16.
    const int r = lane & 15, n = c0 + 4 * (lane >> 4);
    if (r >= rows) return;
    const float xs = QROWS ? row_scale[r] : p.a_scales[r];
    i32x4_t sum = {0, 0, 0, 0};
    for (int i = 0; i < waves; ++i) sum += *reinterpret_cast<const i32x4_t*>(own + i * wave_bytes + lane * 16);
    uint16_t* out = p.y[0] + static_cast<int64_t>(r) * N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < N) out[e] = f32_to_bf16_bits(static_cast<float>(sum[e]) * p.w_scales[0][n + e] * xs);
}

}  // namespace

bool w8_qmv_shape(int rows, int waves, int K, bool quantize, W8QmvShape* out) {
    const int lines = (K + 127) / 128;
    out->rows = rows;
    out->waves = waves;
    out->share = (lines + waves - 1) / waves;
    out->lds = 64 + 64 * kW8QmvWaves + static_cast<size_t>(waves) * std::min(out->share, kLines) * kW8QmvColumns * 128;
    if (quantize) out->lds += static_cast<size_t>(rows) * (K + 16);
    return rows <= (quantize ? kW8QuantizeRows : kW8QmvRows) && out->lds <= 163840 && (!quantize || K / 8 <= kPieces * 64 * waves);
}

hipError_t launch_w8_qmv(const W8QmvShape& s, const W8TileArgs& args, hipStream_t stream) {
    const int blocks = (args.N + kW8QmvColumns - 1) / kW8QmvColumns;
    auto run = [&](auto kernel) {
        if (s.lds > 65536) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(s.lds));
            if (e != hipSuccess) return e;
        }
        W4A16_LAUNCH(kernel, dim3(blocks), dim3(64 * s.waves), s.lds, stream, args, s.share, blocks);
        return hipGetLastError();
    };
    if (!args.x) return run(w8_qmv_kernel<0>);
    return s.rows == 1 ? run(w8_qmv_kernel<1>) : run(w8_qmv_kernel<2>);
}

}  // namespace w4a16
