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
//  * LDS holds stages of BM rows of the left operand and BN rows of the weights.  The 16-byte chunk c
//    of row r lies at c ^ ((r / 2) % 8): sixteen consecutive rows read one chunk from all sixteen
//    16-byte bank groups.
//  * The left operand, and codes that need no decoding, go from memory to LDS directly.  Weights to
//    be decoded are loaded into registers two to four steps ahead, decoded (four instructions per
//    eight values) one step ahead and written to LDS once per workgroup, so that all waves share the
//    decoding.  A step waits only for the loads that it uses (counted, in the order of issue).
//  * kColumns needs, for one output column, eight consecutive contraction values in a lane, while
//    the codes are packed along the output columns.  Decoded rows are staged as they come, from
//    whole 128-byte lines; the operand reads are the transposing ones.  (Bytes exchanged by permutes
//    before the write, from 2-byte loads: 4096 x 9728 x 2560 took 252 us, this 210 in the same tiles.)
//  * Of the 128 bytes, MFMA step j of lane half h takes chunk 4 h + j.  For codes a chunk is one
//    block, so the four scale bytes that a lane needs in a pipeline step are one aligned word of the
//    row's scales.  (Steps of whole 128-byte lines: taking 64 bytes from each of two lines, which also
//    gives such words, is twice the requests to L2; 66 us against 58 at 4096 x 2560 x 9728.)
//  * The weights are the MFMA's row operand, so a lane's results are four consecutive output
//    columns of one row; each wave turns its block through LDS and stores whole 16-byte pieces.
//  * With two weight sets (gate and up) the 32-column blocks of the tile alternate between them, so
//    a lane holds both products of the same element and the activation needs no exchange.
//  * Split-K: slice z takes a contiguous run of steps and writes fp32 partials; the slices are
//    summed in order by a second launch, so results do not depend on timing.
//
// Bound by the matrix cores from some 500 rows on, at the clock that the card keeps under them (2.0 to
// 2.2 GHz at 4096 rows, 2.5 under light work).  Traced on MI355X, 4096 rows x weight rows x values; in
// brackets the rate and the share of a compute unit's busy cycles in which its matrix cores are:
//   kCodes    x 9728 x 2560   69 us (3.0 PF, 49%)     x 2560 x 9728   61 us (3.3 PF, 56%)
//   kRows     x 9728 x 2560  190 us (1.07 PF, 70%)    x 2560 x 9728  184 us (1.11 PF, 72%)
//   kColumns  x 9728 x 2560  201 us (1.01 PF, 61%)
//   kGlu      x 9728 x 2560  322 us for both products (1.27 PF, 71%); kGluGrad 367 us (60%)
// The rest is the L2's latency and traffic (the 16-bit kinds fetch some 300 MB, three to eight times
// what they cannot do without): with the left operand's loads left out kRows took 161 us and kColumns
// 169.  kCodes stages one step ahead in all tiles but 64 x 128, and 608 tiles on 256 compute units
// take three rounds.  Below 500 rows the number of workgroups bounds it (the cost model chooses among
// tiles and splits): kRows of 512 x 9728 x 2560 33 us, of 509 x 2560 x 9728 39 and 4 for the slices'
// sum, kGlu of 512 x 9728 x 2560 54.
#include "mxfp4_device.h"
#include "mxfp4_internal.h"

#include <type_traits>

namespace w4a16 {
namespace {

// All but the last PENDING loads of this wave have arrived, its LDS accesses are done, and all waves
// are here.
template <int PENDING>
__device__ __forceinline__ void loads_done_barrier() {
    static_assert(PENDING <= 63, "the counter of outstanding loads has six bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PENDING) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Keeps the loads before it and after it in this order, and apart.
__device__ __forceinline__ void load_fence() { asm volatile("" ::: "memory"); }

// WHOLE: the rows of scales are whole, aligned pieces of 16 bytes (kCodes) or of 4 (kRows).
template <MxOperands OP, MxEpilogue EPI, int BM, int BN, int WR, int WC, int STAGES, bool WHOLE>
__global__ __launch_bounds__(64 * WR * WC) void mx_tile_kernel(const MxTileArgs p, int tiles_m, int tiles_n) {
    constexpr int NW = WR * WC, NT = 64 * NW;
    constexpr int MI = BM / WR / 32, NI = BN / WC / 32;      // 32 x 32 blocks of a wave
    constexpr bool kCodes = OP == MxOperands::kCodes, kColumns = OP == MxOperands::kColumns;
    constexpr bool kPair = EPI != MxEpilogue::kStore;
    static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "direct loads: whole rows, one chunk order");
    static_assert(!kPair || (NI % 2 == 0 && !kColumns), "both weight sets of an element in one wave");
    constexpr int BC = kPair ? BN / 2 : BN;                  // output columns of the tile

    // one object per stage, so that a direct load into one is not taken for an input of reads of the others
    static_assert(STAGES == 2 || STAGES == 4, "a pair of steps has one parity of stages");
    constexpr bool kDeep = STAGES == 4;
    __shared__ __attribute__((aligned(16))) uint8_t a0[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a1[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t a2[kDeep ? BM * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t a3[kDeep ? BM * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t b0[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b1[BN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t b2[kDeep && kCodes ? BN * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t b3[kDeep && kCodes ? BN * 128 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t sc[kCodes ? 2 * NT * 16 : 16];
    auto a_stage = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value % STAGES;
        if constexpr (i == 0) return a0;
        else if constexpr (i == 1) return a1;
        else if constexpr (i == 2) return a2;
        else return a3;
    };
    // decoded weights are staged one step ahead: two stages
    auto b_stage = [&](auto ic) -> uint8_t* {
        constexpr int i = decltype(ic)::value % (kCodes ? STAGES : 2);
        if constexpr (i == 0) return b0;
        else if constexpr (i == 1) return b1;
        else if constexpr (i == 2) return b2;
        else return b3;
    };

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
        const int pairs = (blocks + 15) / 16;
        t_begin = 2 * static_cast<int>(static_cast<int64_t>(z) * pairs / p.split);
        t_end = min(2 * static_cast<int>(static_cast<int64_t>(z + 1) * pairs / p.split), (blocks + 7) / 8);
    } else {
        // kRows: slices are pairs of steps
        constexpr int unit = OP == MxOperands::kRows ? 2 : 1;
        const int units = (kColumns ? set_steps * p.sets : set_steps + 1) / unit;
        t_begin = unit * static_cast<int>(static_cast<int64_t>(z) * units / p.split);
        t_end = unit * static_cast<int>(static_cast<int64_t>(z + 1) * units / p.split);
    }

    // ---- left operand: direct loads, instruction i of this wave fills rows 8 (wave + NW i) .. + 7
    constexpr int A_LOADS = BM / (8 * NW);
    const int a_chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    const uint32_t a_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * left_row) + 16u * a_chunk;
    auto issue_rows = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t off, int pitch, uint8_t* dst, int t, int step,
                          auto loads) {
        const bool inside = t < t_end && (kCodes ? 8 * step + a_chunk < blocks : 64 * step + 8 * a_chunk < L);
        const uint32_t at = 128u * step;
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
    const uint32_t b_off = static_cast<uint32_t>((8 * wave + (lane >> 3)) * row_codes) + 16u * a_chunk;
    // Decoded weights: a thread takes one block (16 bytes of codes) of every step, unit tid.
    //  kColumns: rows of the step side by side, block u % (BN / 32) of row u / (BN / 32): whole 128-byte
    //    lines; loaded four steps ahead (two: 128 x 128 tiles alone on their units took 0.65 us a step).
    //  kRows: two blocks per row and step would be 32-byte pieces of 128-byte lines, so two steps are
    //    loaded at once, four lanes on the four blocks of a row.  Loads 0 and 1 of a lane are two rows;
    //    lanes 0 and 1 of four keep the first and lanes 2 and 3 the second row for both steps, and get
    //    (DPP quad_perm 2 3 0 1) what the others loaded of it.  The rows' order makes eight lanes' writes
    //    fall into eight different chunks.  A lane's four scale bytes of two steps are one word.
    constexpr bool kRows = OP == MxOperands::kRows;
    static_assert(kCodes || BN * 2 == NT, "one block per thread and step");
    constexpr int ROW_BLOCKS = BN / 32;                       // kColumns: blocks of a row of the tile
    const int quad = lane >> 2, upper = (lane >> 1) & 1;
    auto quad_row = [&](int i) { return 32 * wave + 2 * (i + 2 * (quad & 7)) + (quad >> 3); };
    const int unit_row = kRows ? quad_row(upper) : tid / ROW_BLOCKS;
    const int unit_block = kRows ? lane & 1 : tid % ROW_BLOCKS;
    u32x4_t w_codes[4];                                       // four steps, or two pairs of loads
    uint32_t w_scale[kColumns || !WHOLE ? 4 : 2];
    // (a wave's rows are 32 consecutive ones: one weight set)
    const int own_set = kRows ? set_of(32 * wave) : 0;
    const __amdgpu_buffer_rsrc_t own_codes = own_set ? wr1 : wr0;
    const __amdgpu_buffer_rsrc_t own_scales =
        mx_resource(p.w_scales[own_set] + static_cast<int64_t>(c0) * blocks, columns_left * blocks);
    // kRows: the blocks of steps t and t + 1 (t even) into slot SLOT
    auto load_pair = [&](int t, auto slot) {
        if constexpr (kRows) {
            constexpr int at = decltype(slot)::value;
            const int first = 2 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t co = first + (lane & 3) < blocks
                                        ? static_cast<uint32_t>(column_of(quad_row(i)) * row_codes + 16 * (lane & 3))
                                        : kOutside;
                w_codes[2 * at + i] =
                    __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(own_codes, co, 16 * first, 0));
                load_fence();
            }
            const uint32_t so = static_cast<uint32_t>(column_of(unit_row) * blocks);
            if constexpr (WHOLE) {
                w_scale[at] = __builtin_amdgcn_raw_buffer_load_b32(own_scales, first < blocks ? so : kOutside, first, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w_scale[2 * at + i] = __builtin_amdgcn_raw_buffer_load_b8(
                        own_scales, first + 2 * i + unit_block < blocks ? so + unit_block : kOutside, first + 2 * i, 0);
                    load_fence();
                }
            }
        }
    };
    // kColumns: the blocks of step t into slot SLOT
    auto load_step = [&](int t, auto slot) {
        if constexpr (kColumns) {
            constexpr int at = decltype(slot)::value % 4;
            const int set = p.sets > 1 && t >= set_steps ? 1 : 0;
            const int64_t n = 64 * static_cast<int64_t>(t - set * set_steps);
            const __amdgpu_buffer_rsrc_t cr =
                mx_resource(p.w[set] + n * row_codes + c0 / 2, (L - n) * row_codes - c0 / 2);
            const __amdgpu_buffer_rsrc_t sr =
                mx_resource(p.w_scales[set] + n * blocks + c0 / kMxBlock, (L - n) * blocks - c0 / kMxBlock);
            const bool inside = c0 / kMxBlock + unit_block < blocks;
            w_codes[at] = __builtin_bit_cast(
                u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                             cr, inside ? static_cast<uint32_t>(unit_row * row_codes + 16 * unit_block) : kOutside, 0, 0));
            w_scale[at] = __builtin_amdgcn_raw_buffer_load_b8(
                sr, inside ? static_cast<uint32_t>(unit_row * blocks + unit_block) : kOutside, 0, 0);
        }
    };
    // Decoding and staging a step (its number modulo four), in four parts that the products of the
    // step before are spread over.  kColumns stages rows of BN values as they come; the operand reads
    // transpose them.  16-byte chunk c of row n lies at c ^ (c / 8) % 4 ^ 4 (n % 4) ^ 2 (n % 2):
    // conflict-free for the writes (eight lanes on eight blocks of a row, or on four of two rows) and
    // for reads of 4 rows x 32 columns.
    auto stash_weights = [&](auto ic, auto qc) {
        constexpr int n = decltype(ic)::value, q = decltype(qc)::value;
        uint8_t* dst = b_stage(ic);
        if constexpr (kRows) {
            constexpr int pair = n / 2 % 2, odd = n % 2;
            const uint32_t mine = w_codes[2 * pair + odd][q], other = w_codes[2 * pair + 1 - odd][q];
            const uint32_t moved = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(other), 0x4E, 0xF, 0xF, true));
            const uint32_t w = upper == odd ? mine : moved;
            const uint32_t e = WHOLE ? (w_scale[pair] >> (8 * (2 * odd + unit_block))) & 0xFFu : w_scale[2 * pair * !WHOLE + odd];
            const int c = (4 * unit_block + q) ^ ((unit_row >> 1) & 7);
            *reinterpret_cast<u32x4_t*>(dst + unit_row * 128 + 16 * c) = mx_decode_word(w, mx_scale(e));
        }
        if constexpr (kColumns) {
            constexpr int at = n % 4;
            const int c = (4 * unit_block + (q ^ (unit_block >> 1))) ^ (4 * (unit_row & 3)) ^ (2 * (unit_row & 1));
            *reinterpret_cast<u32x4_t*>(dst + unit_row * (2 * BN) + 16 * c) =
                mx_decode_word(w_codes[at][q], mx_scale(w_scale[at]));
        }
    };

    // ---- scales of both operands (kCodes): thread r < BM + BN keeps row r's next 16 bytes, one
    // load where rows are whole pieces of 16, a byte each elsewhere.  A byte past the row's last
    // block is put to 0 (a finite scale: its codes are zeros).
    static_assert(!kCodes || (BM + BN <= NT && BM % 64 == 0), "one row of scales per thread, one operand per wave");
    constexpr int PAIRS = STAGES / 2;
    u32x4_t s_next[PAIRS];               // of the next pairs of steps
    uint32_t s_bytes[PAIRS][!kCodes || WHOLE ? 1 : 16];
    const bool s_left = kCodes && wave < BM / 64;
    const int s_first = s_left ? m0 : c0;
    const __amdgpu_buffer_rsrc_t s_rows =
        mx_resource((s_left ? p.a_scales : p.w_scales[0]) + static_cast<int64_t>(s_first) * blocks,
                    (static_cast<int64_t>(s_left ? p.M : p.N) - s_first) * blocks);
    const uint32_t s_off = static_cast<uint32_t>((s_left ? tid : tid - BM) * blocks);
    auto load_scales = [&](int window, auto ic) {
        constexpr int pair = decltype(ic)::value / 2 % PAIRS;
        if constexpr (kCodes && WHOLE) {
            s_next[pair] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                     s_rows, 16 * window < blocks ? s_off : kOutside, 16 * window, 0));
        } else if constexpr (kCodes) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s_bytes[pair][e] = __builtin_amdgcn_raw_buffer_load_b8(
                    s_rows, 16 * window + e < blocks ? s_off : kOutside, 16 * window + e, 0);
                load_fence();
            }
        }
    };
    auto stash_scales = [&](int window, auto ic) {
        constexpr int pair = decltype(ic)::value / 2 % PAIRS;
        if constexpr (kCodes) {
            if constexpr (!WHOLE) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    s_next[pair][q] = s_bytes[pair][4 * q] | s_bytes[pair][4 * q + 1] << 8 |
                                      s_bytes[pair][4 * q + 2] << 16 | s_bytes[pair][4 * q + 3] << 24;
            }
            *reinterpret_cast<u32x4_t*>(sc + (window & 1) * NT * 16 + tid * 16) = s_next[pair];
        }
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // Chunk c of this lane's row of a block; rows of a block share (r / 2) % 8.
    const int arow = wr * MI * 32 + (lane & 31), brow = wc * NI * 32 + (lane & 31);
    const int key = (lane >> 1) & 7;
    // kColumns: a transposing read gives lane i of sixteen column i of 4 rows x 16 columns, of which it
    // addresses 4 columns of row i / 4
    const int t_row = 32 * half + ((lane & 15) >> 2);
    const int t_low = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    // The products lag one MFMA step behind the reads, across the barrier too, so that an LDS read has
    // MFMAs to hide under.  Operands of two MFMA steps and scales of two pipeline steps, by parity; zeros
    // at first, for the products that the first pipeline step makes of the one before it.
    u32x4_t af[2][MI], bf[2][NI];
    uint32_t sa[2][MI], sb[2][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) af[1][i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NI; ++i) bf[1][i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[1][i] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) sb[1][i] = 0;
    auto read_scales = [&](int t, auto ic) {
        if constexpr (kCodes) {
            constexpr int par = decltype(ic)::value & 1;
            const uint8_t* s = sc + ((t >> 1) & 1) * NT * 16 + 8 * (t & 1) + 4 * half;
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
            af[j & 1][i] = *reinterpret_cast<const u32x4_t*>(as + i * 4096 + 16 * ((4 * half + j) ^ key));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if constexpr (kColumns) {
                typedef short s16x4_t __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4;
                const int cb = wc * NI + i, a = (lane & 15) >> 2;
                const int chunk = ((4 * cb) ^ (4 * a)) + (t_low ^ ((cb / 2) & 3) ^ (2 * (a & 1)));
                const uint8_t* at = b_stage(ic) + (t_row + 8 * j) * (2 * BN) + 16 * chunk + 8 * (lane & 1);
                // rows 8 (4 half + j) + 0 .. 3 and + 4 .. 7
                const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at));
                const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 4 * 2 * BN));
                bf[j & 1][i] = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                bf[j & 1][i] = *reinterpret_cast<const u32x4_t*>(bs + i * 4096 + 16 * ((4 * half + j) ^ key));
            }
        }
    };
    auto multiply = [&](auto ic, auto jc) {
        constexpr int j = decltype(jc)::value, par = decltype(ic)::value & 1;
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
            issue_rows(wr0, b_off, row_codes, b_stage(ic), t, t, std::integral_constant<int, B_LOADS>{});
    };
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Three = std::integral_constant<int, 3>;
    // Loads of a step: the left operand (and codes) of the step AHEAD of it, then, in some steps, more:
    // kCodes scales in even steps, kRows two steps' weights in odd ones, kColumns weights in each.
    constexpr int AHEAD = STAGES - 1;
    constexpr int kStepLoads = A_LOADS + (kCodes ? B_LOADS : 0);
    constexpr auto more_loads = [](int parity) {
        return kCodes ? (parity == 0 ? (WHOLE ? 1 : 16) : 0) : kRows ? (parity == 1 ? (WHOLE ? 3 : 4) : 0) : 2;
    };
    // loads issued after those that a step of this parity waits for (load_fence keeps each a separate
    // instruction, in this order)
    constexpr auto pending = [more_loads](int parity) {
        int n = more_loads((parity + AHEAD) % 2);
        for (int s = 1; s < AHEAD; ++s) n += kStepLoads + more_loads((parity + s) % 2);
        return n;
    };
    // (all of the first loads are on their way before the first is waited for)
    if constexpr (kCodes) {
        load_scales(t_begin >> 1, Zero{});
        if constexpr (kDeep) load_scales((t_begin >> 1) + 1, Two{});
    } else {
        load_pair(t_begin, Zero{});
        load_step(t_begin, Zero{});
    }
    stage_step(t_begin, Zero{});
    if constexpr (kDeep) {
        stage_step(t_begin + 1, One{});
        stage_step(t_begin + 2, Two{});
    }
    load_pair(t_begin + 2, One{});
    load_step(t_begin + 1, One{});
    load_step(t_begin + 2, Two{});
    load_step(t_begin + 3, Three{});
    stash_scales(t_begin >> 1, Zero{});
    stash_weights(Zero{}, Zero{});
    stash_weights(Zero{}, One{});
    stash_weights(Zero{}, Two{});
    stash_weights(Zero{}, Three{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // step t, whose number modulo four is that of ic
    auto step = [&](int t, auto ic) {
        constexpr int i = decltype(ic)::value;
        using Next = std::integral_constant<int, i + 1>;
        using Ahead = std::integral_constant<int, i + AHEAD>;
        using Before = std::integral_constant<int, i + 1>;                // (parity of step t - 1)
        loads_done_barrier<pending(i % 2)>();
        read_scales(t, ic);
        read(ic, Zero{});
        // every load of this step is issued here, as long as possible before the wait for it
        stage_step(t + AHEAD, Ahead{});
        load_fence();
        if constexpr (kCodes && i % 2 == 0) load_scales((t >> 1) + PAIRS, ic);
        if constexpr (kRows && i % 2 == 1) load_pair(t + 3, std::integral_constant<int, (i + 3) / 2 % 2>{});
        if constexpr (kColumns) load_step(t + 4, ic);
        stash_weights(Next{}, Zero{});
        multiply(Before{}, Three{});          // of step t - 1
        __builtin_amdgcn_sched_barrier(0);
        read(ic, One{});
        stash_weights(Next{}, One{});
        multiply(ic, Zero{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Two{});
        stash_weights(Next{}, Two{});
        multiply(ic, One{});
        __builtin_amdgcn_sched_barrier(0);
        read(ic, Three{});
        if constexpr (kCodes && i % 2 == 1) stash_scales((t >> 1) + 1, Next{});
        stash_weights(Next{}, Three{});
        multiply(ic, Two{});
        __builtin_amdgcn_sched_barrier(0);
    };
    // steps past the end, up to a whole round, have a left operand of zeros
    constexpr int ROUND = kCodes ? STAGES : 4;
    for (int t = t_begin; t < t_end; t += ROUND) {
        step(t, Zero{});
        step(t + 1, One{});
        if constexpr (ROUND == 4) {
            step(t + 2, Two{});
            step(t + 3, Three{});
        }
    }
    multiply(One{}, Three{});

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
    loads_done_barrier<0>();
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

const MxTileShape kMxTiles[kNumMxTiles] = {{128, 128, 4}, {256, 256, 8}, {64, 128, 4}, {192, 256, 8}, {128, 256, 8}};

namespace {

// Stages of the left operand; CODE_STAGES of the form that stages both operands as they come.  Four
// stages cover a latency with three steps of loads, at the cost of a second workgroup beside: 64 x 128
// with decoded weights (64 KB) keeps both, of codes (104 KB) only one fits.  192 x 256 fits four of the left operand and two of decoded weights into 160 KB (4096 x
// 2560 with 9728 values: 198 us with two, 190 with four; kColumns 211 and 208), 256 x 256 does not;
// 128 x 128 gained nothing from them.  128 x 256 has two waves a SIMD where 128 x 128 alone on its compute
// unit has one: 1024 rows of 9728 values on 2560 columns 77 and 61 us, 2048 rows of codes 51 and 43.
template <int BM, int BN, int WR, int WC, int STAGES, int CODE_STAGES>
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
        return whole ? run(mx_tile_kernel<O::kCodes, E::kStore, BM, BN, WR, WC, CODE_STAGES, true>)
                     : run(mx_tile_kernel<O::kCodes, E::kStore, BM, BN, WR, WC, CODE_STAGES, false>);
    }
    if (op == O::kColumns) return run(mx_tile_kernel<O::kColumns, E::kStore, BM, BN, WR, WC, STAGES, true>);
    // words of four scale bytes in every row
    const bool words = args.L % 128 == 0 && ((reinterpret_cast<uintptr_t>(args.w_scales[0]) |
                                              reinterpret_cast<uintptr_t>(args.w_scales[1])) & 3) == 0;
    auto rows = [&](auto ec) {
        constexpr E e = decltype(ec)::value;
        return words ? run(mx_tile_kernel<O::kRows, e, BM, BN, WR, WC, STAGES, true>)
                     : run(mx_tile_kernel<O::kRows, e, BM, BN, WR, WC, STAGES, false>);
    };
    if (epi == E::kGlu) return rows(std::integral_constant<E, E::kGlu>{});
    if (epi == E::kGluGrad) return rows(std::integral_constant<E, E::kGluGrad>{});
    return rows(std::integral_constant<E, E::kStore>{});
}

}  // namespace

hipError_t launch_mx_tile(MxOperands op, MxEpilogue epi, int tile, const MxTileArgs& args, hipStream_t stream) {
    switch (tile) {
        case 0: return launch_shape<128, 128, 2, 2, 2, 2>(op, epi, args, stream);
        case 1: return launch_shape<256, 256, 2, 4, 2, 2>(op, epi, args, stream);
        case 2: return launch_shape<64, 128, 2, 2, 4, 4>(op, epi, args, stream);
        case 3: return launch_shape<192, 256, 2, 4, 4, 2>(op, epi, args, stream);
        case 4: return launch_shape<128, 256, 2, 4, 4, 2>(op, epi, args, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
