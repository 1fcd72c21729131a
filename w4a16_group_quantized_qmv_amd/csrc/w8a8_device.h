// Device helpers of the int8 kernels (gfx950 / CDNA4 only).
//
// v_mfma_i32_32x32x32_i8:  lane l holds row (column) l % 32, sixteen consecutive values 16 (l / 32) ..;
// v_mfma_i32_16x16x64_i8:  row (column) l % 16, values 16 (l / 16) ..;  D as in the bf16 shapes.  Any
// bijection between the instruction's K index and real indices serves both operands.
#pragma once

#include "mxfp4_device.h"

namespace w4a16 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x16_t mfma32_i8(const u32x4_t& a, const u32x4_t& b, const i32x16_t& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ i32x4_t mfma16_i8(const u32x4_t& a, const u32x4_t& b, const i32x4_t& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                                 0);
}

// All but the last PENDING loads of this wave have arrived, its LDS accesses are done, and all waves
// are here.
template <int PENDING>
__device__ __forceinline__ void w8_loads_done_barrier() {
    static_assert(PENDING <= 63, "the counter of outstanding loads has six bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PENDING) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The quantizer's rule for a row whose largest magnitude is a (a NaN counts as such): the factor that
// takes values to codes and the scale that takes them back.  Below 2^-110 a row counts as zeros: the format's
// own bound, a margin above 2^-119 and 2^-121, under which a / 127 is subnormal and 127 / a passes the largest
// fp32 number; a row with an infinity or a NaN gets the scale NaN.  Both divisions are correctly rounded (the compiler's default).
__device__ __forceinline__ void w8_row_scale(float a, float& inverse, float& scale) {
    const bool tiny = a < 0x1p-110f, finite = a < __builtin_inff();
    inverse = tiny || !finite ? 0.f : 127.f / a;
    scale = tiny ? 0.f : finite ? a / 127.f : __builtin_nanf("");
}

// One value's code: the product rounded to fp32, then to the nearest integer, ties to even.  A row with
// the factor 0 (zeros, or not finite) has codes 0.
__device__ __forceinline__ uint32_t w8_code(float x, float inverse) {
    const float v = inverse == 0.f ? 0.f : __builtin_rintf(x * inverse);
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(v, -127.f), 127.f))) & 0xFFu;
}

// Which tile of which expert a workgroup takes.  Rows are clamped to [0, R], whatever the offsets hold.
struct ExpertTile {
    int expert, first, end;     // the expert's rows
    int tm, tn;
    int piece, cut;             // of a tile that is cut into pieces of rows
};

// Tile number `block` of the experts' tiles of BM rows x tiles_n columns of tiles, in an order that gives each XCD
// whole experts where it can; false where there are fewer tiles.  What is left after whole rounds over `cus`
// compute units is cut into two or four pieces (`most` of them) where all of them run at once.  Every wave calls
// it, with all lanes; the result is uniform.
template <int BAND>
__device__ __forceinline__ bool find_expert_tile(const int* __restrict__ offsets, int E, int R, int BM, int tiles_n,
                                                 int cus, int most, int block, ExpertTile& out) {
    const int lane = threadIdx.x & 63;
    const int per = (E + 63) >> 6;
    auto rows_of = [&](int e, int& first, int& end) {
        first = min(max(offsets[e], 0), R);
        end = max(min(max(offsets[e + 1], 0), R), first);
        return (end - first + BM - 1) / BM;
    };
    // (offsets that fall could count rows twice, and past 31 bits: what the grid does not hold is left out)
    const int room = static_cast<int>(gridDim.x);
    int mine = 0, first, end;
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < E) mine = min(mine + rows_of(e, first, end), room);
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        if (lane >= d) sum += v;
    }
    const int64_t all = static_cast<int64_t>(__builtin_amdgcn_readlane(sum, 63)) * tiles_n;
    const int total = static_cast<int>(min(all, static_cast<int64_t>(room)));
    int whole = total;
    out.cut = 1;
    if (most > 1 && total > cus) {
        const int rest = total % cus;
        out.cut = most >= 4 && 4 * rest <= cus ? 4 : 2 * rest <= cus ? 2 : 1;
        if (out.cut > 1) whole = total - rest;
    }
    const int items = whole + (total - whole) * out.cut;
    if (block >= items) return false;
    int work;
    if (block < whole) {
        work = xcd_remap(block, whole);
        out.piece = 0;
        out.cut = 1;
    } else {
        const int item = xcd_remap(block - whole, items - whole);
        work = whole + item / out.cut;
        out.piece = item % out.cut;
    }
    const uint64_t past = __ballot(static_cast<int64_t>(sum) * tiles_n > work);
    const int owner = __builtin_ctzll(past);
    int before = __builtin_amdgcn_readlane(sum - mine, owner);
    for (int i = 0; i < per; ++i) {
        const int e = owner * per + i;
        if (e >= E) break;
        const int tiles = rows_of(e, first, end);
        if (static_cast<int64_t>(before + tiles) * tiles_n > work) {
            out.expert = e;
            out.first = first;
            out.end = end;
            band_order<BAND>(work - before * tiles_n, tiles, tiles_n, out.tm, out.tn);
            return true;
        }
        before += tiles;
    }
    return false;
}

}  // namespace w4a16
