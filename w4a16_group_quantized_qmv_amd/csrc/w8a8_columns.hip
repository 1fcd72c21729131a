// The transposed product of int8 weights, tiled: the input gradient of a projection, of one expert after the
// other's, or of a gated pair.
//
//   dx[r, k] = sum_s sum_n g_s[r, n] w_scale_s[n] w_s[n, k]
//
// The scale belongs to the contracted index, so one of the bf16 operands has to carry it, and is rounded once for
// it.  SCALED: the weights, decoded to bf16(w_scale w), and gradient rows are taken as they come; scaling those
// would take a pass of its own over them.  Else the gradient rows, by the kernel that made them in fp32 (the gated
// pair's), and a weight is its code, exact in bf16: one rounding on the way to dx either way, not two.
//
//  * A pipeline step is 64 rows of the weights, and of every gradient row 64 values (128 bytes).  Gradient rows
//    go from memory to LDS directly: chunk c of row r at c ^ ((r / 2) % 8).
//  * The operand wants, for one output column, eight consecutive contraction values in a lane, while the codes
//    lie along the output columns.  Each thread loads 32 codes of one weight row, some steps ahead, decodes them
//    a step ahead and writes 64 bytes to LDS as they come; the operand reads are the transposing ones.
//    Chunk c of row n lies at c ^ (c / 8) % 4 ^ 4 (n % 4) ^ 2 (n % 2): conflict-free for the writes and for
//    reads of 4 rows x 32 columns.
//  * Split-K (one matrix): slices take runs of steps and write fp32 partials that are summed in order.
#include "w8a8_device.h"
#include "w8a8_internal.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

__device__ __forceinline__ void load_fence() { asm volatile("" ::: "memory"); }

// Eight codes of two words, times a scale or not, as bf16.
template <bool SCALED>
__device__ __forceinline__ u32x4_t decode8(uint32_t lo, uint32_t hi, float scale) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? lo : hi;
        const float a = static_cast<float>(static_cast<int8_t>(w >> (16 * (i & 1))));
        const float b = static_cast<float>(static_cast<int8_t>(w >> (16 * (i & 1) + 8)));
        r[i] = SCALED ? pack_bf16(a * scale, b * scale) : pack_bf16(a, b);
    }
    return r;
}

struct Place {
    int expert, m0, m_end, c0, z;
};
// One object per stage, so that a direct load into one is not taken for an input of reads of the others.
struct Stages {
    uint8_t *a0, *a1, *a2, *a3, *b0, *b1;
};

template <bool EXPERTS, bool SCALED, int MI, int NI, int WR, int WC, int STAGES>
__device__ __forceinline__ void w8_columns(const W8ColumnsArgs& p, const Stages& lds, const Place& place) {
    constexpr int NW = WR * WC, NT = 64 * NW, BM = 32 * MI * WR, BN = 32 * NI * WC;
    static_assert(NW % 2 == 0, "direct loads: one chunk order");
    static_assert(BN * 2 == NT, "32 codes per thread and step");
    static_assert(STAGES == 2 || STAGES == 4, "a round of four steps");
    constexpr bool kDeep = STAGES == 4;
    auto a_stage = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value % STAGES;
        if constexpr (i == 0) return lds.a0;
        else if constexpr (i == 1) return lds.a1;
        else if constexpr (i == 2) return lds.a2;
        else return lds.a3;
    };
    auto b_stage = [&](auto ic) -> uint8_t* { return decltype(ic)::value % 2 ? lds.b1 : lds.b0; };

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / WC, wc = wave % WC;
    const int z = place.z, expert = place.expert, m0 = place.m0, m_end = place.m_end, c0 = place.c0;

    const int N = p.N, K = p.K;                              // contraction, output columns
    const int set_steps = (N + 63) / 64;
    const int steps = set_steps * p.sets;
    const int t_begin = static_cast<int>(static_cast<int64_t>(z) * steps / p.split);
    const int t_end = static_cast<int>(static_cast<int64_t>(z + 1) * steps / p.split);

    // ---- gradient rows
    constexpr int A_LOADS = (BM + 8 * NW - 1) / (8 * NW);     // (rows behind the tile's last are outside the buffer)
    const int own_chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    const int row_bytes = 2 * p.pitch;
    const uint32_t a_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * row_bytes) + 16u * own_chunk;
    const int64_t a_base = static_cast<int64_t>(m0) * p.pitch, a_bytes = static_cast<int64_t>(m_end - m0) * row_bytes;
    const __amdgpu_buffer_rsrc_t ar0 = mx_resource(p.g[0] + a_base, a_bytes);
    const __amdgpu_buffer_rsrc_t ar1 = p.sets > 1 ? mx_resource(p.g[1] + a_base, a_bytes) : ar0;
    auto issue_left = [&](int t, auto ic) {
        const int set = p.sets > 1 && t >= set_steps ? 1 : 0, s = t - set * set_steps;
        const bool inside = t < t_end && 64 * s + 8 * own_chunk < N;
        const uint32_t at = 128u * s;
        const __amdgpu_buffer_rsrc_t r = set ? ar1 : ar0;
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i) {
            uint8_t* to = a_stage(ic) + __builtin_amdgcn_readfirstlane((wave + NW * i) * 1024);
            const uint32_t o = inside ? a_off + static_cast<uint32_t>(8 * NW * i) * static_cast<uint32_t>(row_bytes) : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, o, at, 0, 0);
        }
    };

    // ---- weights: this thread's 32 codes are block unit_block of row unit_row of a step
    constexpr int ROW_BLOCKS = BN / 32, DEPTH = 4;
    const int unit_row = tid / ROW_BLOCKS, unit_block = tid % ROW_BLOCKS;
    u32x4_t codes[DEPTH][2];
    uint32_t scale[DEPTH] = {};
    auto load_step = [&](int t, auto slot) {
        constexpr int at = decltype(slot)::value % DEPTH;
        const int set = p.sets > 1 && t >= set_steps ? 1 : 0;
        const int64_t n = 64 * static_cast<int64_t>(t - set * set_steps), row = static_cast<int64_t>(expert) * N + n;
        // (steps past a slice's end take no weights of the next one: zeros times an infinite one would be NaN)
        const int64_t rows = EXPERTS || t < t_end ? N - n : 0;
        const __amdgpu_buffer_rsrc_t cr = mx_resource(p.w[set] + row * K + c0, rows * K - c0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int column = 32 * unit_block + 16 * i;
            const uint32_t o = c0 + column < K ? static_cast<uint32_t>(unit_row) * static_cast<uint32_t>(K) + column : kOutside;
            codes[at][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(cr, o, 0, 0));
        }
        if constexpr (SCALED) {
            const __amdgpu_buffer_rsrc_t sr = mx_resource(p.w_scales[set] + row, 4 * rows);
            scale[at] = __builtin_amdgcn_raw_buffer_load_b32(sr, 4 * unit_row, 0, 0);
        }
    };
    auto stash = [&](auto ic, auto qc) {
        constexpr int n = decltype(ic)::value, q = decltype(qc)::value, at = n % DEPTH;
        const int c = (4 * unit_block + (q ^ (unit_block >> 1))) ^ (4 * (unit_row & 3)) ^ (2 * (unit_row & 1));
        *reinterpret_cast<u32x4_t*>(b_stage(ic) + unit_row * (2 * BN) + 16 * c) =
            decode8<SCALED>(codes[at][q >> 1][2 * (q & 1)], codes[at][q >> 1][2 * (q & 1) + 1], __uint_as_float(scale[at]));
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const int arow = wr * MI * 32 + (lane & 31), key = (lane >> 1) & 7;
    // A transposing read gives lane i of sixteen column i of 4 rows x 16 columns, of which it addresses 4
    // columns of row i / 4.
    const int t_row = 32 * half + ((lane & 15) >> 2);
    const int t_low = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    // The products lag one MFMA step behind the reads, across the barrier too.
    u32x4_t af[2][MI], bf[2][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) af[1][i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NI; ++i) bf[1][i] = u32x4_t{0, 0, 0, 0};
    auto read = [&](auto ic, auto jc) {
        constexpr int j = decltype(jc)::value;
        const uint8_t* as = a_stage(ic) + arow * 128;
#pragma unroll
        for (int i = 0; i < MI; ++i)
            af[j & 1][i] = *reinterpret_cast<const u32x4_t*>(as + i * 4096 + 16 * ((4 * half + j) ^ key));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            typedef short s16x4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4;
            const int cb = wc * NI + i, a = (lane & 15) >> 2;
            const int chunk = ((4 * cb) ^ (4 * a)) + (t_low ^ ((cb / 2) & 3) ^ (2 * (a & 1)));
            const uint8_t* at = b_stage(ic) + (t_row + 8 * j) * (2 * BN) + 16 * chunk + 8 * (lane & 1);
            // rows 8 (4 half + j) + 0 .. 3 and + 4 .. 7
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at));
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 4 * 2 * BN));
            bf[j & 1][i] = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    };
    auto multiply = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int k = 0; k < NI; ++k)
                acc[i][k] = mfma32x32x16(__builtin_bit_cast(bf16x8_t, bf[j & 1][k]),
                                         __builtin_bit_cast(bf16x8_t, af[j & 1][i]), acc[i][k]);
    };

    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Three = std::integral_constant<int, 3>;
    constexpr int AHEAD = STAGES - 1, MORE = SCALED ? 3 : 2;              // loads of a step beside the gradient rows'
    constexpr int kPending = MORE + (AHEAD - 1) * (A_LOADS + MORE);
    load_step(t_begin, Zero{});
    load_fence();
    issue_left(t_begin, Zero{});
    if constexpr (kDeep) {
        issue_left(t_begin + 1, One{});
        issue_left(t_begin + 2, Two{});
    }
    load_fence();
    load_step(t_begin + 1, One{});
    load_step(t_begin + 2, Two{});
    load_step(t_begin + 3, Three{});
    stash(Zero{}, Zero{});
    stash(Zero{}, One{});
    stash(Zero{}, Two{});
    stash(Zero{}, Three{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    auto step = [&](int t, auto ic) {
        constexpr int i = decltype(ic)::value;
        using Next = std::integral_constant<int, i + 1>;
        w8_loads_done_barrier<kPending>();
        read(ic, Zero{});
        issue_left(t + AHEAD, std::integral_constant<int, i + AHEAD>{});
        load_fence();
        load_step(t + 4, ic);
        load_fence();
        stash(Next{}, Zero{});
        multiply(Three{});                    // of step t - 1
        __builtin_amdgcn_sched_barrier(0);
        read(ic, One{});
        stash(Next{}, One{});
        multiply(Zero{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Two{});
        stash(Next{}, Two{});
        multiply(One{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Three{});
        stash(Next{}, Three{});
        multiply(Two{});
        __builtin_amdgcn_sched_barrier(0);
    };
    // steps past the end, up to a whole round, have a left operand of zeros (branches for what is left of a round made
    // the compiler spill: 32768 rows of a gated pair 1947 us)
    for (int t = t_begin; t < t_end; t += 4) {
        step(t, Zero{});
        step(t + 1, One{});
        step(t + 2, Two{});
        step(t + 3, Three{});
    }
    multiply(Three{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");         // no load into LDS outlives the workgroup

    // ---- epilogue.  Register r of a block: column 8 (r / 4) + 4 half + r % 4, row lane % 32.
    const int row0 = m0 + wr * MI * 32, col0 = c0 + wc * NI * 32;
    if (!EXPERTS && p.split > 1) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = row0 + 32 * i + (lane & 31);
            if (m >= m_end) continue;
            float* out = p.ws + (static_cast<size_t>(z) * p.R + m) * K;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = col0 + 32 * j + 4 * half + 8 * q;
                    if (n < K)                               // (K is a multiple of 16)
                        *reinterpret_cast<f32x4_t*>(out + n) =
                            f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                }
        }
        return;
    }
    constexpr int WCOLS = NI * 32, PITCH = WCOLS * 2 + 16, PIECES = WCOLS / 8;
    static_assert((NW / 2) * 32 * PITCH <= BN * 128, "the waves' regions fit the weight stages");
    w8_loads_done_barrier<0>();
    uint8_t* region = ((wave & 1) ? lds.b1 : lds.b0) + (wave >> 1) * (32 * PITCH);
    const bool wide = (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t* at = reinterpret_cast<uint32_t*>(region + (lane & 31) * PITCH + (32 * j + 8 * q + 4 * half) * 2);
                at[0] = pack_bf16(acc[i][j][4 * q], acc[i][j][4 * q + 1]);
                at[1] = pack_bf16(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
            }
        wave_lds_fence();
#pragma unroll
        for (int u = 0; u < 32 * PIECES / 64; ++u) {
            const int r = (64 * u + lane) / PIECES, c = (64 * u + lane) % PIECES;
            const int m = row0 + 32 * i + r, n = col0 + 8 * c;
            if (m >= m_end || n >= K) continue;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(region + r * PITCH + 16 * c);
            uint16_t* out = p.y + static_cast<size_t>(m) * K + n;
            if (wide) {
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out));   // (not read again here)
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
            }
        }
        wave_lds_fence();
    }
}

// The tile's height by the rows that are there.
template <bool EXPERTS, bool SCALED, int MI, int NI, int WR, int WC, int STAGES>
__device__ __forceinline__ void w8_columns_of_height(const W8ColumnsArgs& p, const Stages& lds, const Place& place) {
    if constexpr (MI > 1) {
        if (place.m_end - place.m0 <= 32 * (MI - 1) * WR) {
            w8_columns_of_height<EXPERTS, SCALED, MI - 1, NI, WR, WC, STAGES>(p, lds, place);
            return;
        }
    }
    w8_columns<EXPERTS, SCALED, MI, NI, WR, WC, STAGES>(p, lds, place);
}

template <bool EXPERTS, bool SCALED, int MI, int NI, int WR, int WC, int STAGES>
__global__ __launch_bounds__(64 * WR * WC) void w8_columns_kernel(const W8ColumnsArgs p, int height, int tiles_m, int tiles_n,
                                                                  int whole, int cut) {
    constexpr int BN = 32 * NI * WC;
    constexpr int ROWS = (32 * MI * WR + 8 * WR * WC - 1) / (8 * WR * WC) * (8 * WR * WC);    // whole loads of all waves
    __shared__ __attribute__((aligned(16))) uint8_t a0[ROWS * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a1[ROWS * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a2[STAGES > 2 ? ROWS * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t a3[STAGES > 2 ? ROWS * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t b0[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b1[BN * 128];
    const Stages lds{a0, a1, a2, a3, b0, b1};
    Place place{0, 0, 0, 0, 0};
    if constexpr (EXPERTS) {
        ExpertTile tile;
        if (!find_expert_tile<kBandM>(p.offsets, p.E, p.R, height, tiles_n, p.cus, cut, blockIdx.x, tile)) return;
        place.expert = tile.expert;
        const int rows = (height + tile.cut - 1) / tile.cut, m = tile.first + tile.tm * height;
        place.m0 = m + tile.piece * rows;
        place.m_end = min(min(tile.end, m + height), place.m0 + rows);
        if (place.m0 >= place.m_end) return;
        place.c0 = tile.tn * BN;
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
        place.c0 = tn * BN;
        if (place.m0 >= place.m_end) return;
    }
    w8_columns_of_height<EXPERTS, SCALED, MI, NI, WR, WC, STAGES>(p, lds, place);
}

}  // namespace

// 64 x 128, two of four waves a compute unit; 128 x 256, whose waves have all rows of 32 columns, four stages; and 256 x
// 256.  A step costs at least 0.8 us, so lower tiles bring nothing (2048 x 4096 x 2560 in 96 rows 60 us, in 128 61).
const W8TileShape kW8ColumnTiles[kNumW8ColumnTiles] = {{64, 128, 4, 64}, {128, 256, 8, 32}, {256, 256, 8, 64}};

namespace {

template <int MI, int NI, int WR, int WC, int STAGES>
hipError_t launch_shape(const W8ColumnsArgs& args, hipStream_t stream) {
    constexpr int BN = 32 * NI * WC;
    const int BM = args.height > 0 ? std::min(args.height, 32 * MI * WR) : 32 * MI * WR;
    const int tiles_n = (args.K + BN - 1) / BN;
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
    if (!args.w_scales[0]) return run(w8_columns_kernel<true, false, MI, NI, WR, WC, STAGES>);
    return args.offsets ? run(w8_columns_kernel<true, true, MI, NI, WR, WC, STAGES>)
                        : run(w8_columns_kernel<false, true, MI, NI, WR, WC, STAGES>);
}

}  // namespace

hipError_t launch_w8_columns(int tile, const W8ColumnsArgs& args, hipStream_t stream) {
    switch (tile) {
        case 0: return launch_shape<1, 2, 2, 2, 4>(args, stream);
        case 1: return launch_shape<4, 1, 1, 8, 4>(args, stream);
        case 2: return launch_shape<4, 2, 2, 4, 2>(args, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
