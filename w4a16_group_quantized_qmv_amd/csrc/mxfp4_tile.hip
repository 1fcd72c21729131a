// MXFP4 products on the matrix cores, tiled: the weight-only product and its transpose (bf16 rows
// by decoded weights), the product of two MXFP4 operands (scaled MFMA), and the gated block's
// epilogues.
//
//   kCodes     D[m, n] = sum_k 2^(ea + ew) a[m, k] w[n, k]       both operands as they are stored
//   kRows      D[m, n] = sum_k x[m, k] w[n, k]                   w decoded to bf16 (exact)
//   kColumns   D[m, k] = sum_s sum_n g_s[m, n] w_s[n, k]         w decoded and transposed on the way
//   kGlu       h = silu(D_gate) * D_up
//   kGluGrad   s = sigmoid(D_gate);  dup = dh D_gate s;  dgate = dh D_up s (1 + D_gate (1 - s))
//
// One frame serves all of them, because every staged row is 128 bytes per pipeline step: 64 bf16
// values or 256 codes.
//  * LDS holds BM rows of the left operand and BN rows of the weights, two stages.  The 16-byte
//    chunk c of row r lies at c ^ ((r / 2) % 8): sixteen consecutive rows read one chunk from all
//    sixteen 16-byte bank groups.  kColumns also folds r / 16 in, since its writes go four rows apart.
//  * The left operand, and codes that need no decoding, go from memory to LDS directly.  Weights
//    to be decoded are loaded into registers one step ahead, decoded (four instructions per eight
//    values) and written to LDS once per workgroup, so the decoding is shared by all waves.
//  * kColumns needs, for one output column, eight consecutive contraction values in a lane, while
//    the codes are packed along the output columns.  A thread takes 8 weight rows x 4 columns
//    (2 bytes of each row), decodes pairs of columns and exchanges halves with 16 byte permutes.
//  * Of the 128 bytes, MFMA step j of lane half h takes chunk 4 h + j.  For codes a chunk is one
//    block, and a pair of pipeline steps covers 16 blocks so distributed that a lane's four scale
//    bytes per step are one aligned word: step i, half h, MFMA j is block 8 h + 4 i + j.
//  * The weights are the MFMA's row operand, so a lane's results are four consecutive output
//    columns of one row; each wave turns its block through LDS and stores whole 16-byte pieces.
//  * With two weight sets (gate and up) the 32-column blocks of the tile alternate between them, so
//    a lane holds both products of the same element and the activation needs no exchange.
//  * Split-K: slice z takes a contiguous run of steps and writes fp32 partials; the slices are
//    summed in order by a second launch, so results do not depend on timing.
#include "mxfp4_device.h"
#include "mxfp4_internal.h"

#include <type_traits>

namespace w4a16 {
namespace {

constexpr uint32_t kOutside = 0x80000000u;   // a buffer offset that no resource here reaches

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_resource(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFFll ? 0x7FFFFFFFll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(n), 0x00020000);
}

// All of this wave's loads have arrived and all waves are here.
__device__ __forceinline__ void loads_done_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// WHOLE (kCodes): rows of scales are whole, aligned pieces of 16 bytes.
template <MxOperands OP, MxEpilogue EPI, int BM, int BN, int WR, int WC, bool WHOLE>
__global__ __launch_bounds__(64 * WR * WC) void mx_tile_kernel(const MxTileArgs p, int tiles_m, int tiles_n) {
    constexpr int NW = WR * WC, NT = 64 * NW;
    constexpr int MI = BM / WR / 32, NI = BN / WC / 32;      // 32 x 32 blocks of a wave
    constexpr bool kCodes = OP == MxOperands::kCodes, kColumns = OP == MxOperands::kColumns;
    constexpr bool kPair = EPI != MxEpilogue::kStore;
    static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "direct loads: whole rows, one chunk order");
    static_assert(!kPair || (NI % 2 == 0 && !kColumns), "both weight sets of an element in one wave");
    constexpr int BC = kPair ? BN / 2 : BN;                  // output columns of the tile

    // one object per stage, so that a direct load into one is not taken for an input of reads of the other
    __shared__ __attribute__((aligned(16))) uint8_t a0[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a1[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b0[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b1[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t sc[kCodes ? 2 * (BM + BN) * 16 : 16];
    auto a_stage = [&](auto ic) -> uint8_t* { if constexpr (decltype(ic)::value == 0) return a0; else return a1; };
    auto b_stage = [&](auto ic) -> uint8_t* { if constexpr (decltype(ic)::value == 0) return b0; else return b1; };

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / WC, wc = wave % WC;

    const int tiles = tiles_m * tiles_n;
    const int work = xcd_remap(blockIdx.x, tiles * p.split);
    const int z = work / tiles;
    int tm, tn;
    band_order<kBandM>(work - z * tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, c0 = tn * BC;

    // The contraction: blocks of a row of codes, and pipeline steps.  kColumns runs over the
    // weight sets one after the other.
    const int L = p.L;
    const int blocks = (kColumns ? p.N : L) / kMxBlock;      // blocks of one weight row
    const int row_codes = blocks * 16;                       // bytes of one weight row
    const int left_row = static_cast<int>(p.pitch);          // bytes of one row of the left operand
    const int set_steps = (L + 63) / 64;                     // bf16 operands
    int t_begin, t_end;
    if constexpr (kCodes) {
        const int rest = blocks % 16, windows = (blocks + 15) / 16;
        const int w0 = static_cast<int>(static_cast<int64_t>(z) * windows / p.split);
        const int w1 = static_cast<int>(static_cast<int64_t>(z + 1) * windows / p.split);
        t_begin = 2 * w0;
        t_end = 2 * w1 - (w1 == windows && rest > 0 && rest <= 4 ? 1 : 0);
    } else {
        const int steps = kColumns ? set_steps * p.sets : set_steps;
        t_begin = static_cast<int>(static_cast<int64_t>(z) * steps / p.split);
        t_end = static_cast<int>(static_cast<int64_t>(z + 1) * steps / p.split);
    }

    // ---- left operand: direct loads, instruction i of this wave fills rows 8 (wave + NW i) .. + 7
    constexpr int A_LOADS = BM / (8 * NW);
    const int a_chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    uint32_t a_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * left_row) +
                     (kCodes ? 128u * (a_chunk >> 2) + 16u * (a_chunk & 3) : 16u * a_chunk);
    auto issue_rows = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t off, int pitch, uint8_t* dst, int t, int step,
                          auto loads) {
        bool inside;
        uint32_t at;
        if constexpr (kCodes) {
            inside = 16 * (t >> 1) + 4 * (t & 1) + 8 * (a_chunk >> 2) + (a_chunk & 3) < blocks;
            at = 256u * (t >> 1) + 64u * (t & 1);
        } else {
            inside = 64 * step + 8 * a_chunk < L;
            at = 128u * step;
        }
#pragma unroll
        for (int i = 0; i < decltype(loads)::value; ++i) {
            uint8_t* to = dst + __builtin_amdgcn_readfirstlane((wave + NW * i) * 1024);
            const uint32_t o = inside ? off + static_cast<uint32_t>(8 * NW * i) * static_cast<uint32_t>(pitch) : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, o, at, 0, 0);
        }
    };
    const __amdgpu_buffer_rsrc_t ar0 =
        mx_resource(static_cast<const uint8_t*>(p.a[0]) + static_cast<int64_t>(m0) * left_row,
                    static_cast<int64_t>(p.M - m0) * left_row);
    const __amdgpu_buffer_rsrc_t ar1 =
        kColumns && p.sets > 1 ? mx_resource(static_cast<const uint8_t*>(p.a[1]) + static_cast<int64_t>(m0) * left_row,
                                             static_cast<int64_t>(p.M - m0) * left_row)
                               : ar0;
    auto issue_left = [&](int t, auto ic) {
        const int set = kColumns && p.sets > 1 && t >= set_steps ? 1 : 0;
        issue_rows(set ? ar1 : ar0, a_off, left_row, a_stage(ic), t, t - set * set_steps,
                   std::integral_constant<int, A_LOADS>{});
    };

    // ---- weights
    // row r of the tile -> weight set and column
    auto set_of = [](int r) { return kPair ? (r >> 5) & 1 : 0; };
    auto column_of = [](int r) { return kPair ? (r >> 6) * 32 + (r & 31) : r; };
    const int64_t columns_left = p.N - c0;
    auto set_base = [&](int s) { return mx_resource(p.w[s] + static_cast<int64_t>(c0) * row_codes, columns_left * row_codes); };
    const __amdgpu_buffer_rsrc_t wr0 = set_base(0), wr1 = kPair ? set_base(1) : wr0;
    // kCodes: direct loads as for the left operand (one weight set)
    constexpr int B_LOADS = kCodes ? BN / (8 * NW) : 1;
    static_assert(!(kCodes && kPair), "the pair decodes its weights");
    const uint32_t b_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * row_codes) +
                           128u * (a_chunk >> 2) + 16u * (a_chunk & 3);
    // kRows: a thread takes whole blocks.  A wave has both blocks of 32 rows, two lanes a row,
    // the even rows in its first half: eight lanes' writes then fall into eight different chunks.
    constexpr int UNITS = OP == MxOperands::kRows ? BN * 2 / NT : 1;
    static_assert(OP != MxOperands::kRows || BN * 2 % NT == 0, "whole units");
    auto unit_row = [&](int i) { return 32 * (wave + NW * i) + (lane & 30) + half; };
    u32x4_t w_codes[2][UNITS];           // of two pipeline steps, by parity
    uint32_t w_scale[2][UNITS];
    // kColumns: 8 rows x 4 columns of the step
    constexpr int GROUP_LANES = kColumns ? BN / 4 : 64;      // threads across the tile's columns
    static_assert(!kColumns || GROUP_LANES * 8 == NT, "one 8 x 4 unit per thread");
    const int t_rows = tid / GROUP_LANES, t_col = 4 * (tid % GROUP_LANES);
    uint16_t t_codes[2][8];
    uint32_t t_scale[2];
    auto load_weights = [&](int t, auto ic) {
        constexpr int par = decltype(ic)::value;
        if constexpr (OP == MxOperands::kRows) {
            const int blk = 2 * t + (lane & 1);
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int r = unit_row(i);
                const int c = column_of(r);
                // (a wave's units are 32 consecutive rows: one weight set)
                const int s = __builtin_amdgcn_readfirstlane(set_of(r));
                const uint32_t co = blk < blocks ? static_cast<uint32_t>(c * row_codes + 16 * (lane & 1)) : kOutside;
                w_codes[par][i] = __builtin_bit_cast(
                    u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(s ? wr1 : wr0, co, 32 * t, 0));
                const __amdgpu_buffer_rsrc_t sr =
                    mx_resource(p.w_scales[s] + static_cast<int64_t>(c0) * blocks, columns_left * blocks);
                const uint32_t so = blk < blocks ? static_cast<uint32_t>(c * blocks + (lane & 1)) : kOutside;
                w_scale[par][i] = __builtin_amdgcn_raw_buffer_load_b8(sr, so, 2 * t, 0);
            }
        }
        if constexpr (kColumns) {
            const int set = p.sets > 1 && t >= set_steps ? 1 : 0;
            const int64_t n = 64 * static_cast<int64_t>(t - set * set_steps);
            const __amdgpu_buffer_rsrc_t cr =
                mx_resource(p.w[set] + n * row_codes + c0 / 2, (L - n) * row_codes - c0 / 2);
            const __amdgpu_buffer_rsrc_t sr =
                mx_resource(p.w_scales[set] + n * blocks + c0 / kMxBlock, (L - n) * blocks - c0 / kMxBlock);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t_codes[par][i] = __builtin_amdgcn_raw_buffer_load_b16(
                    cr, static_cast<uint32_t>((8 * t_rows + i) * row_codes + t_col / 2), 0, 0);
            // lane l of eight holds the scale of row l % 8; they are handed round below
            t_scale[par] = __builtin_amdgcn_raw_buffer_load_b8(
                sr, static_cast<uint32_t>((8 * t_rows + (lane & 7)) * blocks + t_col / kMxBlock), 0, 0);
        }
    };
    // decoding and staging, in four parts that the products of a step are spread over
    uint32_t t_pairs[8][2];    // kColumns: rows, column pairs
    auto stash_weights = [&](auto ic, auto qc) {
        constexpr int q = decltype(qc)::value, par = decltype(ic)::value;
        uint8_t* dst = b_stage(ic);
        if constexpr (OP == MxOperands::kRows) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int r = unit_row(i);
                const int c = (4 * (lane & 1) + q) ^ ((r >> 1) & 7);
                *reinterpret_cast<u32x4_t*>(dst + r * 128 + 16 * c) = mx_decode_word(w_codes[par][i][q], mx_scale(w_scale[par][i]));
            }
        }
        if constexpr (kColumns) {
            auto row = [&](auto rc) {
                constexpr int i = decltype(rc)::value;
                const float s = mx_scale(__builtin_amdgcn_ds_swizzle(static_cast<int>(t_scale[par]), (i << 5) | 0x18));
                t_pairs[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(t_codes[par][i], s, 0));
                t_pairs[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(t_codes[par][i], s, 1));
            };
            if constexpr (q < 2) {
                row(std::integral_constant<int, 4 * (q & 1)>{});
                row(std::integral_constant<int, 4 * (q & 1) + 1>{});
                row(std::integral_constant<int, 4 * (q & 1) + 2>{});
                row(std::integral_constant<int, 4 * (q & 1) + 3>{});
            } else {
#pragma unroll
                for (int k = 2 * (q & 1); k < 2 * (q & 1) + 2; ++k) {
                    u32x4_t out;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[i] = __builtin_amdgcn_perm(t_pairs[2 * i + 1][k >> 1], t_pairs[2 * i][k >> 1],
                                                       (k & 1) ? 0x07060302u : 0x05040100u);
                    const int r = t_col + k;
                    const int c = t_rows ^ (((r >> 1) ^ (r >> 4)) & 7);
                    *reinterpret_cast<u32x4_t*>(dst + r * 128 + 16 * c) = out;
                }
            }
        }
    };

    // ---- scales of both operands (kCodes): thread r < BM + BN keeps row r's next 16 bytes, one
    // load where rows are whole pieces of 16, a byte each elsewhere.  A byte past the row's last
    // block is put to 0 (a finite scale: its codes are zeros).
    static_assert(!kCodes || (BM + BN == NT && BM % 64 == 0), "one row of scales per thread, one operand per wave");
    u32x4_t s_next = {0, 0, 0, 0};
    uint32_t s_bytes[!kCodes || WHOLE ? 1 : 16];
    const bool s_left = kCodes && wave < BM / 64;
    const int s_first = s_left ? m0 : c0;
    const __amdgpu_buffer_rsrc_t s_rows =
        mx_resource((s_left ? p.a_scales : p.w_scales[0]) + static_cast<int64_t>(s_first) * blocks,
                    (static_cast<int64_t>(s_left ? p.M : p.N) - s_first) * blocks);
    const uint32_t s_off = static_cast<uint32_t>((s_left ? tid : tid - BM) * blocks);
    auto load_scales = [&](int window) {
        if constexpr (kCodes && WHOLE) {
            s_next = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                     s_rows, 16 * window < blocks ? s_off : kOutside, 16 * window, 0));
        } else if constexpr (kCodes) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s_bytes[e] = __builtin_amdgcn_raw_buffer_load_b8(
                    s_rows, 16 * window + e < blocks ? s_off : kOutside, 16 * window + e, 0);
        }
    };
    auto stash_scales = [&](int window) {
        if constexpr (kCodes) {
            if constexpr (!WHOLE) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    s_next[q] = s_bytes[4 * q] | s_bytes[4 * q + 1] << 8 | s_bytes[4 * q + 2] << 16 |
                                s_bytes[4 * q + 3] << 24;
            }
            *reinterpret_cast<u32x4_t*>(sc + (window & 1) * (BM + BN) * 16 + tid * 16) = s_next;
        }
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // chunk c of this lane's row of block b: rows of a block share (r / 2) % 8; kColumns adds 2 b
    const int arow = wr * MI * 32 + (lane & 31), brow = wc * NI * 32 + (lane & 31);
    const int akey = (lane >> 1) & 7;
    const int bkey = kColumns ? (akey ^ ((lane >> 4) & 1)) : akey;
    // operands of two MFMA steps (by parity) and the scales of two pipeline steps; zeros at first, for
    // the products that the first pipeline step makes of the step before it
    u32x4_t af[2][MI], bf[2][NI];
    uint32_t sa[2][MI], sb[2][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        af[1][i] = u32x4_t{0, 0, 0, 0};
        sa[1][i] = 0;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        bf[1][i] = u32x4_t{0, 0, 0, 0};
        sb[1][i] = 0;
    }
    auto read_scales = [&](int t, auto ic) {
        if constexpr (kCodes) {
            constexpr int par = decltype(ic)::value;
            const uint8_t* s = sc + ((t >> 1) & 1) * (BM + BN) * 16 + 8 * half + 4 * (t & 1);
#pragma unroll
            for (int i = 0; i < MI; ++i) sa[par][i] = *reinterpret_cast<const uint32_t*>(s + (arow + 32 * i) * 16);
#pragma unroll
            for (int j = 0; j < NI; ++j) sb[par][j] = *reinterpret_cast<const uint32_t*>(s + (BM + brow + 32 * j) * 16);
        }
    };
    auto read = [&](auto ic, auto jc) {
        constexpr int j = decltype(jc)::value;
        const uint8_t* as = a_stage(ic) + arow * 128;
        const uint8_t* bs = b_stage(ic) + brow * 128;
#pragma unroll
        for (int i = 0; i < MI; ++i)
            af[j & 1][i] = *reinterpret_cast<const u32x4_t*>(as + i * 4096 + 16 * ((4 * half + j) ^ akey));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            // row / 16 of block wc * NI + i: 2 (wc NI + i) + lane / 16 % 2
            const int k = kColumns ? (bkey ^ ((2 * (wc * NI + i)) & 7)) : bkey;
            bf[j & 1][i] = *reinterpret_cast<const u32x4_t*>(bs + i * 4096 + 16 * ((4 * half + j) ^ k));
        }
    };
    auto multiply = [&](auto ic, auto jc) {
        constexpr int j = decltype(jc)::value, par = decltype(ic)::value;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int k = 0; k < NI; ++k) {
                if constexpr (kCodes)
                    acc[i][k] = mx_mfma32<j>(bf[j & 1][k], sb[par][k], af[j & 1][i], sa[par][i], acc[i][k]);
                else
                    acc[i][k] = mfma32x32x16(__builtin_bit_cast(bf16x8_t, bf[j & 1][k]),
                                             __builtin_bit_cast(bf16x8_t, af[j & 1][i]), acc[i][k]);
            }
    };

    // ---- pipeline: while step t is multiplied, step t + 1 goes to the other stage and the codes
    // (scales) of the step (pair of steps) after it into registers.  Nothing in a step is
    // conditional: loads past the contraction's end read zeros, and what lies past a slice's end is
    // staged and left.  (A branch after the products lets the compiler sink them past the next
    // step's reads, at twice the registers.)
    auto stage_step = [&](int t, auto ic) {
        issue_left(t, ic);
        if constexpr (kCodes)
            issue_rows(wr0, b_off, row_codes, b_stage(ic), t, 0, std::integral_constant<int, B_LOADS>{});
    };
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Three = std::integral_constant<int, 3>;
    if constexpr (kCodes) {
        load_scales(t_begin >> 1);
        stash_scales(t_begin >> 1);
    } else {
        load_weights(t_begin, Zero{});
        stash_weights(Zero{}, Zero{});
        stash_weights(Zero{}, One{});
        stash_weights(Zero{}, Two{});
        stash_weights(Zero{}, Three{});
        load_weights(t_begin + 1, One{});
    }
    stage_step(t_begin, Zero{});
    auto step = [&](int t, auto ic, auto nc) {
        loads_done_barrier();
        read_scales(t, ic);
        read(ic, Zero{});
        // every load of this step is issued here, a whole step before the wait for it
        stage_step(t + 1, nc);
        if constexpr (!kCodes)
            load_weights(t + 2, ic);
        else if constexpr (decltype(ic)::value == 0)
            load_scales((t >> 1) + 1);
        stash_weights(nc, Zero{});
        multiply(nc, Three{});          // of step t - 1
        __builtin_amdgcn_sched_barrier(0);
        read(ic, One{});
        stash_weights(nc, One{});
        multiply(ic, Zero{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Two{});
        stash_weights(nc, Two{});
        multiply(ic, One{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Three{});
        // t is even exactly when ic is the even stage: slices start at a pair of steps
        if constexpr (kCodes && decltype(ic)::value == 1) stash_scales((t >> 1) + 1);
        stash_weights(nc, Three{});
        multiply(ic, Two{});
        __builtin_amdgcn_sched_barrier(0);
    };
    int t = t_begin;
    for (; t + 2 <= t_end; t += 2) {
        step(t, Zero{}, One{});
        step(t + 1, One{}, Zero{});
    }
    if (t < t_end) {
        step(t, Zero{}, One{});
        multiply(Zero{}, Three{});
    } else {
        multiply(One{}, Three{});
    }

    // ---- epilogue.  Register r of a block: column 8 (r / 4) + 4 half + r % 4, row lane % 32.
    const int row0 = m0 + wr * MI * 32;
    if (EPI != MxEpilogue::kGluGrad && p.split > 1) {
        // partials [set][split][M][N]
        const bool wide = p.N % 4 == 0;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int m = row0 + 32 * i + (lane & 31);
            if (m >= p.M) continue;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int s = kPair ? j & 1 : 0;
                const int n0 = c0 + column_of(brow - (lane & 31) + 32 * j) + 4 * half;
                float* out = p.ws + ((static_cast<size_t>(s) * p.split + z) * p.M + m) * p.N;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = n0 + 8 * q;
                    if (wide && n < p.N) {
                        *reinterpret_cast<f32x4_t*>(out + n) = f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                                      acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < p.N) out[n + e] = acc[i][j][4 * q + e];
                    }
                }
            }
        }
        return;
    }
    // A wave's region: 32 rows of its columns, rows 16 bytes longer against bank conflicts.
    constexpr int WCOLS = kPair ? NI * 16 : NI * 32;
    constexpr int PITCH = WCOLS * 2 + 16;
    static_assert((NW / 2) * 32 * PITCH <= BN * 128, "the waves' regions fit the weight stages");
    loads_done_barrier();
    uint8_t* region = ((wave & 1) ? b1 : b0) + (wave >> 1) * (32 * PITCH);
    const int col0 = c0 + (kPair ? wc * NI * 16 : wc * NI * 32);
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
    auto flush = [&](uint16_t* y, int i) {
        const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
        wave_lds_fence();
        for_pieces([&](int r, int c) {
            const int m = row0 + 32 * i + r, n = col0 + 8 * c;
            if (m >= p.M || n >= p.N) return;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(region + r * PITCH + 16 * c);
            uint16_t* out = y + static_cast<size_t>(m) * p.N + n;
            if (wide) {
                *reinterpret_cast<u32x4_t*>(out) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < p.N) out[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
            }
        });
        wave_lds_fence();
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if constexpr (EPI == MxEpilogue::kStore) {
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    put(j, q, pack_bf16(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                        pack_bf16(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
            flush(p.y[0], i);
        } else if constexpr (EPI == MxEpilogue::kGlu) {
#pragma unroll
            for (int j = 0; j < NI / 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float g = acc[i][2 * j][4 * q + e];
                        h[e] = g * mx_sigmoid(g) * acc[i][2 * j + 1][4 * q + e];
                    }
                    put(j, q, pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]));
                }
            flush(p.y[0], i);
        } else {
            // dh through the region to the lanes that hold its elements' products
            const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dh) & 15) == 0;
            for_pieces([&](int r, int c) {
                const int m = row0 + 32 * i + r, n = col0 + 8 * c;
                u32x4_t v = {0, 0, 0, 0};
                if (m < p.M && n < p.N) {
                    const uint16_t* in = p.dh + static_cast<size_t>(m) * p.N + n;
                    if (wide) {
                        v = load16(in);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < p.N) v[e >> 1] |= static_cast<uint32_t>(in[e]) << (16 * (e & 1));
                    }
                }
                *reinterpret_cast<u32x4_t*>(region + r * PITCH + 16 * c) = v;
            });
            wave_lds_fence();
#pragma unroll
            for (int j = 0; j < NI / 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t* at =
                        reinterpret_cast<const uint32_t*>(region + (lane & 31) * PITCH + (32 * j + 8 * q + 4 * half) * 2);
                    const uint32_t d[2] = {at[0], at[1]};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float dh = bf16_bits_to_f32(static_cast<uint16_t>(d[e >> 1] >> (16 * (e & 1))));
                        const float g = acc[i][2 * j][4 * q + e], u = acc[i][2 * j + 1][4 * q + e];
                        const float s = mx_sigmoid(g);
                        acc[i][2 * j][4 * q + e] = dh * u * s * (1.f + g * (1.f - s));
                        acc[i][2 * j + 1][4 * q + e] = dh * g * s;
                    }
                }
            wave_lds_fence();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int j = 0; j < NI / 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x16_t& v = acc[i][2 * j + s];
                        put(j, q, pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 2], v[4 * q + 3]));
                    }
                flush(p.y[s], i);
            }
        }
    }
}

}  // namespace

const MxTileShape kMxTiles[kNumMxTiles] = {{128, 128, 4}, {256, 256, 8}};

namespace {

template <int BM, int BN, int WR, int WC>
hipError_t launch_shape(MxOperands op, MxEpilogue epi, const MxTileArgs& args, hipStream_t stream) {
    const int bc = epi == MxEpilogue::kStore ? BN : BN / 2;
    const int tiles_m = (args.M + BM - 1) / BM, tiles_n = (args.N + bc - 1) / bc;
    const dim3 grid(static_cast<uint32_t>(tiles_m) * tiles_n * args.split), block(64 * WR * WC);
    auto run = [&](auto kernel) {
        W4A16_LAUNCH(kernel, grid, block, 0, stream, args, tiles_m, tiles_n);
        return hipGetLastError();
    };
    using O = MxOperands;
    using E = MxEpilogue;
    if (op == O::kCodes) {
        const bool whole = args.L % 512 == 0 && ((reinterpret_cast<uintptr_t>(args.a_scales) |
                                                  reinterpret_cast<uintptr_t>(args.w_scales[0])) & 15) == 0;
        return whole ? run(mx_tile_kernel<O::kCodes, E::kStore, BM, BN, WR, WC, true>)
                     : run(mx_tile_kernel<O::kCodes, E::kStore, BM, BN, WR, WC, false>);
    }
    if (op == O::kColumns) return run(mx_tile_kernel<O::kColumns, E::kStore, BM, BN, WR, WC, true>);
    if (epi == E::kGlu) return run(mx_tile_kernel<O::kRows, E::kGlu, BM, BN, WR, WC, true>);
    if (epi == E::kGluGrad) return run(mx_tile_kernel<O::kRows, E::kGluGrad, BM, BN, WR, WC, true>);
    return run(mx_tile_kernel<O::kRows, E::kStore, BM, BN, WR, WC, true>);
}

}  // namespace

hipError_t launch_mx_tile(MxOperands op, MxEpilogue epi, int tile, const MxTileArgs& args, hipStream_t stream) {
    switch (tile) {
        case 0: return launch_shape<128, 128, 2, 2>(op, epi, args, stream);
        case 1: return launch_shape<256, 256, 2, 4>(op, epi, args, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
