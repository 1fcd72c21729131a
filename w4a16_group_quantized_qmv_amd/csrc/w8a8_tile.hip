// Products of int8 rows by int8 rows on the matrix cores, tiled: one matrix, or one per expert with
// ragged row counts, and the gated block's epilogues.
//
//   P[m, n] = sum_k a[m, k] w[n, k]  in int32, exact (K <= 131056)      D = P w_scale[n] a_scale[m] in fp32
//   kStore    y = bf16(D), or P as a partial of a split contraction
//   kGlu      h = silu(D_gate) D_up
//   kGluGrad  s = sigmoid(D_gate);  dup = dh D_gate s;  dgate = dh D_up s (1 + D_gate (1 - s)), and both times
//             their columns' weight scales, what the product with the codes for dx takes
//
//  * A pipeline step is 128 bytes of every row of the tile, moved from memory to LDS directly.  The
//    16-byte chunk c of row r lies at c ^ ((r / 2) % 8), so sixteen consecutive rows read one chunk from
//    all sixteen 16-byte bank groups.  Chunks past the contraction's end, and rows past the tile's last,
//    are loaded from outside the buffers, as zeros.
//  * Of the 128 bytes, MFMA j of lane half h takes chunk 4 h + j for both operands.
//  * With two weight sets the 32-column blocks of the tile alternate between them, so a lane holds both
//    products of the same element.
//  * Experts: every workgroup finds its tile from the experts' offsets (the host does not know them).
//    The grid holds the most tiles that R rows in E pieces can make, and what is left over ends at once.
//    Rows are gathered by the loads themselves: a lane's row offset is its token's.
#include "w8a8_device.h"
#include "w8a8_internal.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

// What a workgroup works on: rows [m0, m_end) of the expert's (BM of them at most), columns from c0, slice z.
struct Place {
    int expert, m0, m_end, c0, z;
};
// Two to four stages of the left operand's and the weights' rows.  One object per stage, so that a direct load into
// one is not taken for an input of reads of the others.
struct Stages {
    uint8_t *a0, *a1, *a2, *a3, *b0, *b1, *b2, *b3;
};

// One tile of 32 MI WR rows and 32 NI WC rows of weights.
template <W8Epilogue EPI, bool EXPERTS, int MI, int NI, int WR, int WC, int STAGES>
__device__ __forceinline__ void w8_tile(const W8TileArgs& p, const Stages& lds, const Place& place) {
    constexpr int NW = WR * WC, BM = 32 * MI * WR, BN = 32 * NI * WC;
    constexpr bool kPair = EPI != W8Epilogue::kStore;
    static_assert(NW % 2 == 0 && BN % (8 * NW) == 0, "direct loads: whole rows, one chunk order");
    static_assert(!kPair || NI % 2 == 0, "both weight sets of an element in one wave");
    static_assert(STAGES >= 2 && STAGES <= 4, "stages");
    auto a_stage = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value % STAGES;
        if constexpr (i == 0) return lds.a0;
        else if constexpr (i == 1) return lds.a1;
        else if constexpr (i == 2) return lds.a2;
        else return lds.a3;
    };
    auto b_stage = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value % STAGES;
        if constexpr (i == 0) return lds.b0;
        else if constexpr (i == 1) return lds.b1;
        else if constexpr (i == 2) return lds.b2;
        else return lds.b3;
    };

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave / WC, wc = wave % WC;
    const int z = place.z, expert = place.expert, m0 = place.m0, m_end = place.m_end, c0 = place.c0;

    // The contraction in chunks of 16 codes, and this slice's pipeline steps.
    const int K = p.K, chunks = K / kW8Chunk;
    const int steps = (chunks + 7) / 8;
    const int t_begin = static_cast<int>(static_cast<int64_t>(z) * steps / p.split);
    const int t_end = static_cast<int>(static_cast<int64_t>(z + 1) * steps / p.split);

    // ---- left operand: direct load i of this wave fills rows 8 (wave + NW i) .. + 7 of a stage
    // (rows behind the tile's last are read from outside the buffer)
    constexpr int A_LOADS = (BM + 8 * NW - 1) / (8 * NW), B_LOADS = BN / (8 * NW);
    const int own_chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    const bool gather = EXPERTS && p.tokens != nullptr;
    auto source_row = [&](int m) {       // the row of a that output row m takes; -1 for none
        if (m >= m_end) return -1;
        if (!gather) return m;
        const int t = p.tokens[m];
        return t >= 0 && t < p.T ? t : -1;
    };
    const int base = gather ? 0 : m0;
    const int64_t left_rows = (gather ? p.T : m_end) - static_cast<int64_t>(base);
    const __amdgpu_buffer_rsrc_t ar = mx_resource(p.a + static_cast<int64_t>(base) * K, left_rows * K);
    uint32_t a_off[A_LOADS];
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
        const int m = source_row(m0 + 8 * (wave + NW * i) + (lane >> 3));
        a_off[i] = m < 0 ? kOutside : static_cast<uint32_t>(m - base) * static_cast<uint32_t>(K) + 16u * own_chunk;
    }
    // ---- weights: row r of the tile is column column_of(r), of a pair in weight set (r / 32) % 2
    auto column_of = [](int r) { return kPair ? (r >> 6) * 32 + (r & 31) : r; };
    const int64_t w_base = (static_cast<int64_t>(expert) * p.N + c0) * K, w_bytes = static_cast<int64_t>(p.N - c0) * K;
    const __amdgpu_buffer_rsrc_t wr0 = mx_resource(p.w[0] + w_base, w_bytes);
    const __amdgpu_buffer_rsrc_t wr1 = kPair ? mx_resource(p.w[1] + w_base, w_bytes) : wr0;
    uint32_t b_off[B_LOADS];
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i)
        b_off[i] = static_cast<uint32_t>(column_of(8 * (wave + NW * i) + (lane >> 3))) * static_cast<uint32_t>(K) +
                   16u * own_chunk;
    auto stage_step = [&](int t, auto ic) {
        const bool inside = t < t_end && 8 * t + own_chunk < chunks;
        const uint32_t at = 128u * t;
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i) {
            uint8_t* to = a_stage(ic) + __builtin_amdgcn_readfirstlane((wave + NW * i) * 1024);
            const uint32_t o = inside ? a_off[i] : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, to, 16, o, at, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < B_LOADS; ++i) {
            uint8_t* to = b_stage(ic) + __builtin_amdgcn_readfirstlane((wave + NW * i) * 1024);
            const uint32_t o = inside ? b_off[i] : kOutside;
            const __amdgpu_buffer_rsrc_t r = kPair && (((wave + NW * i) >> 2) & 1) ? wr1 : wr0;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, o, at, 0, 0);
        }
    };

    i32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    // Chunk c of this lane's row of a block; rows of a block share (r / 2) % 8.
    const int arow = wr * MI * 32 + (lane & 31), brow = wc * NI * 32 + (lane & 31);
    const int key = (lane >> 1) & 7;
    // The products lag one MFMA step behind the reads, across the barrier too, so that an LDS read has
    // MFMAs to hide under.  Operands of two MFMA steps, by parity; zeros at first, for the products that
    // the first pipeline step makes of the one before it.
    u32x4_t af[2][MI], bf[2][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) af[1][i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NI; ++i) bf[1][i] = u32x4_t{0, 0, 0, 0};
    auto read = [&](auto ic, auto jc) {
        constexpr int j = decltype(jc)::value;
        const uint8_t* as = a_stage(ic) + arow * 128;
        const uint8_t* bs = b_stage(ic) + brow * 128;
#pragma unroll
        for (int i = 0; i < MI; ++i)
            af[j & 1][i] = *reinterpret_cast<const u32x4_t*>(as + i * 4096 + 16 * ((4 * half + j) ^ key));
#pragma unroll
        for (int i = 0; i < NI; ++i)
            bf[j & 1][i] = *reinterpret_cast<const u32x4_t*>(bs + i * 4096 + 16 * ((4 * half + j) ^ key));
    };
    auto multiply = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int k = 0; k < NI; ++k) acc[i][k] = mfma32_i8(bf[j & 1][k], af[j & 1][i], acc[i][k]);
    };

    // ---- pipeline: while step t is multiplied, the steps up to t + STAGES - 1 are on their way.  Loads
    // past the contraction's end read zeros, so nothing in a step is conditional.
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Three = std::integral_constant<int, 3>;
    constexpr int AHEAD = STAGES - 1;
    constexpr int kPending = (AHEAD - 1) * (A_LOADS + B_LOADS);
    stage_step(t_begin, Zero{});
    if constexpr (STAGES > 2) stage_step(t_begin + 1, One{});
    if constexpr (STAGES > 3) stage_step(t_begin + 2, Two{});
    auto step = [&](int t, auto ic) {
        constexpr int i = decltype(ic)::value;
        w8_loads_done_barrier<kPending>();
        read(ic, Zero{});
        // every load of this step is issued here, as long as possible before the wait for it
        stage_step(t + AHEAD, std::integral_constant<int, i + AHEAD>{});
        multiply(Three{});                    // of step t - 1
        __builtin_amdgcn_sched_barrier(0);
        read(ic, One{});
        multiply(Zero{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Two{});
        multiply(One{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Three{});
        multiply(Two{});
        __builtin_amdgcn_sched_barrier(0);
    };
    int t = t_begin;
    for (; t + STAGES <= t_end; t += STAGES) {
        step(t, Zero{});
        step(t + 1, One{});
        if constexpr (STAGES > 2) step(t + 2, Two{});
        if constexpr (STAGES > 3) step(t + 3, Three{});
    }
    // what is left of a round
    if (t < t_end) step(t, Zero{});
    if constexpr (STAGES > 2)
        if (t + 1 < t_end) step(t + 1, One{});
    if constexpr (STAGES > 3)
        if (t + 2 < t_end) step(t + 2, Two{});
    multiply(Three{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // no load into LDS outlives the workgroup

    // ---- epilogue.  Register r of a block: column 8 (r / 4) + 4 half + r % 4, row lane % 32.
    const int row0 = m0 + wr * MI * 32;
    const int col0 = c0 + (kPair ? wc * NI * 16 : wc * NI * 32);      // this wave's first output column
    if (EPI == W8Epilogue::kStore && !EXPERTS && p.split > 1) {
        const bool wide = p.N % 4 == 0;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = row0 + 32 * i + (lane & 31);
            if (m >= m_end) continue;
            int* out = p.ws + (static_cast<size_t>(z) * p.R + m) * p.N;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = col0 + 32 * j + 4 * half + 8 * q;
                    if (wide && n < p.N) {
                        *reinterpret_cast<i32x4_t*>(out + n) =
                            i32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < p.N) out[n + e] = acc[i][j][4 * q + e];
                    }
                }
        }
        return;
    }
    // A wave's region: 32 rows of its columns, rows 16 bytes longer against bank conflicts.
    constexpr int WCOLS = kPair ? NI * 16 : NI * 32;
    constexpr int PITCH = WCOLS * 2 + 16;
    static_assert((NW / 2) * 32 * PITCH <= BN * 128, "the waves' regions fit the weight stages");
    w8_loads_done_barrier<0>();
    uint8_t* region = ((wave & 1) ? lds.b1 : lds.b0) + (wave >> 1) * (32 * PITCH);
    constexpr int PIECES = WCOLS / 8;                        // 16-byte pieces of a row
    auto for_pieces = [&](auto body) {
#pragma unroll
        for (int u = 0; u < 32 * PIECES / 64; ++u) {
            const int r = (64 * u + lane) / PIECES, c = (64 * u + lane) % PIECES;
            body(r, c);
        }
    };
    auto put = [&](int j, int q, uint32_t lo, uint32_t hi) {
        uint32_t* at = reinterpret_cast<uint32_t*>(region + (lane & 31) * PITCH + (32 * j + 8 * q + 4 * half) * 2);
        at[0] = lo;
        at[1] = hi;
    };
    // Rows of `width` columns.  What is not read again here leaves the L2 to the operands (streamed): 32768 rows by
    // experts of 1216 x 2560 148 us without, 131 with, the same tensors again (from memory 149 and 147); of 2560 x 1216
    // from memory 168 and 158.
    auto flush = [&](uint16_t* y, int i, int width, auto streamed) {
        const bool wide = width % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
        wave_lds_fence();
        for_pieces([&](int r, int c) {
            const int m = row0 + 32 * i + r, n = col0 + 8 * c;
            if (m >= m_end || n >= width) return;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(region + r * PITCH + 16 * c);
            uint16_t* out = y + static_cast<size_t>(m) * width + n;
            if (wide) {
                if constexpr (decltype(streamed)::value) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out));
                else *reinterpret_cast<u32x4_t*>(out) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < width) out[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
            }
        });
        wave_lds_fence();
    };
    // the scales of this lane's columns (columns past the last read 0) and rows
    constexpr int BLOCKS = kPair ? NI / 2 : NI, SETS = kPair ? 2 : 1;
    float column_scale[SETS][BLOCKS][16];
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        const __amdgpu_buffer_rsrc_t r = mx_resource(p.w_scales[s] + static_cast<int64_t>(expert) * p.N + col0,
                                                     4 * (static_cast<int64_t>(p.N) - col0));
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                column_scale[s][j][e] = __uint_as_float(
                    __builtin_amdgcn_raw_buffer_load_b32(r, 4u * (32 * j + 8 * (e >> 2) + 4 * half + (e & 3)), 0, 0));
    }
    // dh of all blocks is on its way before the first is used
    constexpr int LOADS = 32 * PIECES / 64;
    u32x4_t dh[EPI == W8Epilogue::kGluGrad ? MI : 1][LOADS];
    if constexpr (EPI == W8Epilogue::kGluGrad) {
        const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dh) & 15) == 0;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int u = 0; u < LOADS; ++u) {
                const int m = row0 + 32 * i + (64 * u + lane) / PIECES, n = col0 + 8 * ((64 * u + lane) % PIECES);
                dh[i][u] = u32x4_t{0, 0, 0, 0};
                if (m < m_end && n < p.N) {
                    const uint16_t* in = p.dh + static_cast<size_t>(m) * p.N + n;
                    if (wide) {
                        dh[i][u] = load16(in);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < p.N) dh[i][u][e >> 1] |= static_cast<uint32_t>(in[e]) << (16 * (e & 1));
                    }
                }
            }
    }
    float row_scale[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = source_row(row0 + 32 * i + (lane & 31));
        row_scale[i] = m < 0 ? 0.f : p.a_scales[m];
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if constexpr (EPI == W8Epilogue::kStore) {
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = static_cast<float>(acc[i][j][4 * q + e]) * column_scale[0][j][4 * q + e] * row_scale[i];
                    put(j, q, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                }
            flush(p.y[0], i, p.N, std::true_type{});
        } else {
            if constexpr (EPI == W8Epilogue::kGluGrad) {
                // dh through the region to the lanes that hold its elements' products
#pragma unroll
                for (int u = 0; u < LOADS; ++u)
                    *reinterpret_cast<u32x4_t*>(region + (64 * u + lane) / PIECES * PITCH + 16 * ((64 * u + lane) % PIECES)) = dh[i][u];
                wave_lds_fence();
            }
            uint32_t more[3][BLOCKS][4][2];              // kGluGrad: what goes through the region after dgate
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t* at =
                        reinterpret_cast<const uint32_t*>(region + (lane & 31) * PITCH + (32 * j + 8 * q + 4 * half) * 2);
                    uint32_t d[2] = {0, 0};
                    if constexpr (EPI == W8Epilogue::kGluGrad) {
                        d[0] = at[0];
                        d[1] = at[1];
                    }
                    float v[4], w[4], sv[4], sw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float gs = column_scale[0][j][4 * q + e], us = column_scale[SETS - 1][j][4 * q + e];
                        const float g = static_cast<float>(acc[i][2 * j][4 * q + e]) * gs * row_scale[i];
                        const float u = static_cast<float>(acc[i][2 * j + 1][4 * q + e]) * us * row_scale[i];
                        const float s = mx_sigmoid(g);
                        if constexpr (EPI == W8Epilogue::kGlu) {
                            v[e] = g * s * u;
                        } else {
                            const float h = bf16_bits_to_f32(static_cast<uint16_t>(d[e >> 1] >> (16 * (e & 1))));
                            v[e] = h * u * s * (1.f + g * (1.f - s));
                            w[e] = h * g * s;
                            sv[e] = v[e] * gs;
                            sw[e] = w[e] * us;
                        }
                    }
                    put(j, q, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                    if constexpr (EPI == W8Epilogue::kGluGrad) {
                        more[0][j][q][0] = pack_bf16(w[0], w[1]);
                        more[0][j][q][1] = pack_bf16(w[2], w[3]);
                        more[1][j][q][0] = pack_bf16(sv[0], sv[1]);
                        more[1][j][q][1] = pack_bf16(sv[2], sv[3]);
                        more[2][j][q][0] = pack_bf16(sw[0], sw[1]);
                        more[2][j][q][1] = pack_bf16(sw[2], sw[3]);
                    }
                }
            flush(p.y[0], i, p.N, std::true_type{});
            if constexpr (EPI == W8Epilogue::kGluGrad) {
                // the scaled gradients' rows are padded: there the products, and so the gradients, are zeros
                const int padded = (p.N + 7) / 8 * 8;
#pragma unroll
                for (int o = 0; o < 3; ++o) {
#pragma unroll
                    for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) put(j, q, more[o][j][q][0], more[o][j][q][1]);
                    if (o == 0) flush(p.y[1], i, p.N, std::true_type{});
                    else flush(p.scaled[o - 1], i, padded, std::false_type{});
                }
            }
        }
    }
}

// The tile's height by the rows that are there: of a shorter one less is loaded and multiplied.
template <W8Epilogue EPI, bool EXPERTS, int MI, int NI, int WR, int WC, int STAGES>
__device__ __forceinline__ void w8_tile_of_height(const W8TileArgs& p, const Stages& lds, const Place& place) {
    constexpr int LESS = MI - 1;
    if constexpr (LESS > 0) {
        if (place.m_end - place.m0 <= 32 * LESS * WR) {
            w8_tile_of_height<EPI, EXPERTS, LESS, NI, WR, WC, STAGES>(p, lds, place);
            return;
        }
    }
    w8_tile<EPI, EXPERTS, MI, NI, WR, WC, STAGES>(p, lds, place);
}

template <W8Epilogue EPI, bool EXPERTS, int MI, int NI, int WR, int WC, int STAGES>
__global__ __launch_bounds__(64 * WR * WC) void w8_tile_kernel(const W8TileArgs p, int height, int tiles_m, int tiles_n,
                                                               int whole, int cut) {
    constexpr int BN = 32 * NI * WC, BC = EPI != W8Epilogue::kStore ? BN / 2 : BN;
    constexpr int ROWS = (32 * MI * WR + 8 * WR * WC - 1) / (8 * WR * WC) * (8 * WR * WC);    // whole loads of all waves
    __shared__ __attribute__((aligned(16))) uint8_t a0[ROWS * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a1[ROWS * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a2[STAGES > 2 ? ROWS * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t a3[STAGES > 3 ? ROWS * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t b0[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b1[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b2[STAGES > 2 ? BN * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t b3[STAGES > 3 ? BN * 128 : 16];
    const Stages lds{a0, a1, a2, a3, b0, b1, b2, b3};
    Place place{0, 0, 0, 0, 0};
    if constexpr (EXPERTS) {
        ExpertTile tile;
        if (!find_expert_tile<kBandM>(p.offsets, p.E, p.R, height, tiles_n, p.cus, cut, blockIdx.x, tile)) return;
        place.expert = tile.expert;
        const int rows = (height + tile.cut - 1) / tile.cut, m = tile.first + tile.tm * height;
        place.m0 = m + tile.piece * rows;
        place.m_end = min(min(tile.end, m + height), place.m0 + rows);
        if (place.m0 >= place.m_end) return;
        place.c0 = tile.tn * BC;
    } else {
        // the first `whole` workgroups take whole tiles, the others tiles cut into `cut` pieces of rows
        const int tiles = tiles_m * tiles_n;
        int work = blockIdx.x, piece = 0;
        if (work < whole) {
            work = xcd_remap(work, whole);
        } else {
            const int rest = xcd_remap(work - whole, gridDim.x - whole);
            work = whole + rest / cut;
            piece = rest % cut;
        }
        place.z = work / tiles;
        int tm, tn;
        band_order<kBandM>(work - place.z * tiles, tiles_m, tiles_n, tm, tn);
        const int rows = blockIdx.x < static_cast<unsigned>(whole) ? height : (height + cut - 1) / cut;
        place.m0 = tm * height + piece * rows;
        place.m_end = min(min(p.R, (tm + 1) * height), place.m0 + rows);
        place.c0 = tn * BC;
        if (place.m0 >= place.m_end) return;
    }
    w8_tile_of_height<EPI, EXPERTS, MI, NI, WR, WC, STAGES>(p, lds, place);
}

}  // namespace

// Where they lead (sweeps of every form; one or two workgroups fit a compute unit):
//   128 x 128  two of four waves a compute unit: middle sizes (2048 x 4096 x 2560 25.8 us; 256 x 256 33)
//   256 x 256  most operations a byte: large ones (4096 x 9728 x 2560 96 us; 128 x 256 104, 128 x 128 112)
//    64 x 128  two a compute unit, three stages: few rows (gated halves of 16 tokens, 64 experts, weights from memory 70
//              us; with four stages and one a compute unit 80, 128 x 128 79)
//   128 x 256  three stages: between those (512 x 9728 x 2560 20.5 us)
//    64 x 256  three stages: few rows of many experts (509 tokens' gated halves 83 us; 128 x 128 91, 64 x 128 97)
//   128 x 128  of eight waves, four stages, one a compute unit: slices of a long contraction with weights from memory
//              (509 x 2560 x 9728 in three slices 23 us, 64 x 128 in one 37; again from the caches 21 and 26); not paired
const W8TileShape kW8Tiles[kNumW8Tiles] = {{128, 128, 4, 64}, {256, 256, 8, 64}, {64, 128, 4, 64}, {128, 256, 8, 64}, {64, 256, 8, 64}, {128, 128, 8, 64}};

namespace {

template <int MI, int NI, int WR, int WC, int STAGES>
hipError_t launch_shape(W8Epilogue epi, const W8TileArgs& args, hipStream_t stream) {
    constexpr int BN = 32 * NI * WC;
    const int BM = args.height > 0 ? std::min(args.height, 32 * MI * WR) : 32 * MI * WR;
    const int bc = epi == W8Epilogue::kStore ? BN : BN / 2;
    const int tiles_n = (args.N + bc - 1) / bc;
    // with experts every one of them may end inside a tile, but none has a tile without a row
    const int tiles_m = args.offsets ? static_cast<int>(std::min<int64_t>(args.R, args.R / BM + args.E)) : (args.R + BM - 1) / BM;
    const int tiles = tiles_m * tiles_n * args.split, cut = std::max(args.cut, 1);
    // (experts: the kernel counts the tiles and cuts, into at most cus pieces)
    const int whole = cut > 1 && !args.offsets ? tiles / args.cus * args.cus : tiles;
    const int more = args.offsets ? (cut > 1 ? args.cus : 0) : (tiles - whole) * (cut - 1);
    const dim3 grid(static_cast<uint32_t>(tiles + more)), block(64 * WR * WC);
    auto run = [&](auto kernel) {
        W4A16_LAUNCH(kernel, grid, block, 0, stream, args, BM, tiles_m, tiles_n, whole, cut);
        return hipGetLastError();
    };
    using E = W8Epilogue;
    if (!args.offsets) return run(w8_tile_kernel<E::kStore, false, MI, NI, WR, WC, STAGES>);
    if (epi != E::kStore && NI % 2 != 0) return hipErrorInvalidValue;
    if constexpr (NI % 2 == 0) {
        if (epi == E::kGlu) return run(w8_tile_kernel<E::kGlu, true, MI, NI, WR, WC, STAGES>);
        if (epi == E::kGluGrad) return run(w8_tile_kernel<E::kGluGrad, true, MI, NI, WR, WC, STAGES>);
    }
    return run(w8_tile_kernel<E::kStore, true, MI, NI, WR, WC, STAGES>);
}

}  // namespace

hipError_t launch_w8_tile(W8Epilogue epi, int tile, const W8TileArgs& args, hipStream_t stream) {
    switch (tile) {
        case 0: return launch_shape<2, 2, 2, 2, 2>(epi, args, stream);      // 128 x 128, 4 waves
        case 1: return launch_shape<4, 2, 2, 4, 2>(epi, args, stream);      // 256 x 256, 8 waves
        case 2: return launch_shape<1, 2, 2, 2, 3>(epi, args, stream);      // 64 x 128, 4 waves
        case 3: return launch_shape<2, 2, 2, 4, 3>(epi, args, stream);      // 128 x 256, 8 waves
        case 4: return launch_shape<1, 2, 2, 4, 3>(epi, args, stream);      // 64 x 256, 8 waves
        case 5: return launch_shape<2, 1, 2, 4, 4>(epi, args, stream);      // 128 x 128, 8 waves
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
