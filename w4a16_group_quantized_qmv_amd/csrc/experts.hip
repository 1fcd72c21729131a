// The router of a mixture of experts and the combination of the experts' outputs, with their gradients.
//
//   route     the top_k largest logits of a token (equal ones: the lowest expert first), their softmax p, and a
//             counting sort of the (token, expert) pairs by expert, then by token
//   backward  with c = sum_j p_j dw_j:  dlogit_e = p_e (dw_e - c), dw_e = 0 for an expert that was not chosen
//   combine   out[t] = sum_j w[t, j] y[row(t, j)]
//   backward  dy[row(t, j)] = w[t, j] dout[t],   dw[t, j] = <dout[t], y[row(t, j)]>
//
// A token takes an expert at most once, so the pairs of 64 tokens are one 64-bit mask per expert: its number of
// bits is the expert's count, and the bits below a token's are the rank of its pair.  The masks are built with
// LDS atomics whose order does not matter, so a call repeats bit for bit.
//
// Bound by latency up to some thousand tokens, the router up to 64 in one launch of one workgroup (5 x 60: 3.2 us).  32767 x
// 256 bf16, eight of them: choice 14 us (17 MB; a chain of one load, eight rounds and a barrier, two workgroups a compute
// unit), scan 4.1, placing 6.1, backward 9.5 (36 MB, 3.8 TB/s).
#include "device_common.h"
#include "mxfp4_device.h"
#include "w4a16.h"
#include "w8a8_internal.h"

#include <type_traits>

namespace w4a16 {
namespace {

constexpr int kTokens = 64;            // tokens of one mask
constexpr int kRouteWaves = 16;

__device__ __forceinline__ float load_logit(const void* logits, bool fp32, int64_t i) {
    return fp32 ? static_cast<const float*>(logits)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(logits)[i]);
}

// A float's bits as an unsigned number of the same order; zeros of both signs are equal.  Minus infinity and NaN
// get 0: they are never chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -__builtin_inff())) return 0u;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

struct RouteArgs {
    const void* logits;
    float* weights;
    int* experts;
    int* positions;
    int* tokens;
    int* offsets;
    int* counts;           // [blocks][E]: first the blocks' counts, then the counts before each block
    int* totals;           // [E]
    int64_t T;
    int E, top_k, blocks;
    bool fp32, renormalize;
};

// Sixteen lanes are a row of the DPP: rotations by 8, 4, 2 and 1 reduce over it, and leave the result in each.
template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, false));
}
template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f) {
    v = f(v, row_rotate<8>(v));
    v = f(v, row_rotate<4>(v));
    v = f(v, row_rotate<2>(v));
    return f(v, row_rotate<1>(v));
}

// The same over the LANES of a token, 16 or all 64.
template <int LANES, typename F>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, F f) {
    v = row_reduce(v, f);
    if constexpr (LANES == 64) {
        auto row = [&](int l) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)); };
        v = f(f(row(0), row(16)), f(row(32), row(48)));
    }
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    return __uint_as_float(lanes_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
    return __uint_as_float(lanes_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

// The logits of a token on its lanes, PER of each: WIDE (E = 16 PER, sixteen lanes) in pieces of 16 bytes (or all PER,
// where those are fewer), neighbours on neighbouring lanes, else one by one.
template <int PER, bool WIDE, bool FP32, int LANES = 16>
__device__ __forceinline__ int expert_of(int lane, int i) {
    constexpr int PIECE = !WIDE ? 1 : PER < (FP32 ? 4 : 8) ? PER : FP32 ? 4 : 8;
    return (lane + LANES * (i / PIECE)) * PIECE + i % PIECE;
}

template <int PER, bool WIDE, bool FP32, int LANES = 16>
__device__ __forceinline__ void load_row(const void* logits, int64_t token, int E, int lane, float (&v)[PER]) {
    static_assert(!WIDE || LANES == 16, "pieces are for sixteen lanes");
    if constexpr (WIDE) {
        constexpr int WORDS = PER * (FP32 ? 4 : 2) / 4;
        const uint32_t* in = static_cast<const uint32_t*>(logits) + token * 16 * WORDS;
        uint32_t w[WORDS];
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const u32x4_t q = load16(in + 4 * (lane + 16 * i));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * i + e] = q[e];
            }
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = in[lane * WORDS + i];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            v[i] = __uint_as_float(FP32 ? w[i * WORDS / PER] : (i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<PER, false, FP32, LANES>(lane, i);
            v[i] = e < E ? load_logit(logits, FP32, token * E + e) : -__builtin_inff();
        }
    }
}

// The chosen experts by rounds over whole keys: of equal ones the lowest.  Lane j gets the j-th.
template <int PER, bool WIDE, int LANES>
__device__ __forceinline__ int choose_exactly(const RouteArgs& p, int64_t token, int lane, bool& nan) {
    uint32_t key[PER];
    {
        float v[PER];
        load_row<PER, WIDE, true, LANES>(p.logits, token, p.E, lane, v);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            nan |= v[i] != v[i];
            key[i] = order_key(v[i]);
        }
    }
    int expert = -1;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0, at = 0xFFFFu;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        best = lanes_reduce<LANES>(best, [](uint32_t a, uint32_t b) { return max(a, b); });
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == best) at = expert_of<PER, WIDE, true, LANES>(lane, i);
        at = lanes_reduce<LANES>(at, [](uint32_t a, uint32_t b) { return min(a, b); });
        if (lane == j && best != 0) expert = at;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (expert_of<PER, WIDE, true, LANES>(lane, i) == static_cast<int>(at)) key[i] = 0;
    }
    return expert;
}

// The same by keys with a number: the expert's, from the largest down, takes the low bits of a logit's key, so that one
// number decides.  With keys k_i and the last one chosen c, k_i - c modulo 2^32 is largest for the largest key below c: a
// round is a subtraction and a maximum for each, and nothing is struck out.  The low 16 bits of a bf16 logit are free.  Of
// an fp32 logit the lowest bits are lost; where two keys in a row differ in nothing else, the token is chosen exactly.
template <int PER, bool WIDE, bool FP32, int LANES>
__device__ __forceinline__ int choose(const RouteArgs& p, int64_t token, int lane, bool& nan) {
    constexpr uint32_t LOW = FP32 ? LANES * PER - 1 : 0xFFFFu;
    static_assert((PER & (PER - 1)) == 0 && LANES * PER <= 65536, "the low bits hold an expert's number");
    uint32_t key[PER];
    {
        float v[PER];
        load_row<PER, WIDE, FP32, LANES>(p.logits, token, p.E, lane, v);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            nan |= v[i] != v[i];
            const uint32_t k = order_key(v[i]);
            key[i] = k == 0 ? 0 : (k & ~LOW) | (LOW - static_cast<uint32_t>(expert_of<PER, WIDE, FP32, LANES>(lane, i)));
        }
    }
    int expert = -1;
    uint32_t last = 0;                     // (2^32: above all keys)
    bool unsure = false;
    const int rounds = FP32 ? min(p.top_k + 1, p.E) : p.top_k;
    for (int j = 0; j < rounds; ++j) {
        uint32_t below = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) below = max(below, key[i] - last);
        below = lanes_reduce<LANES>(below, [](uint32_t a, uint32_t b) { return max(a, b); });
        const uint32_t best = below + last;
        if (best == 0) break;              // (the same on all the token's lanes) nothing is left
        if (FP32) unsure |= j > 0 && (best ^ last) <= LOW;
        if (lane == j && j < p.top_k) expert = LOW - (best & LOW);
        last = best;
    }
    if (FP32 && unsure) expert = choose_exactly<PER, WIDE, LANES>(p, token, lane, nan);
    return expert;
}

// One token by LANES lanes: lane j < top_k gets the j-th chosen expert (-1 for none) and its weight.
template <int PER, bool WIDE, bool FP32, int LANES>
__device__ __forceinline__ void select(const RouteArgs& p, int64_t token, int lane, int& expert, float& weight) {
    bool nan = false;
    // (of up to 256 fp32 logits exactly at once: 32768 x 128 19.3 us, by numbers 20.7; bf16 17.4 and 17.1, x 256 23.0 and 21.9)
    if constexpr (FP32 && LANES == 16 && PER <= 16) expert = choose_exactly<PER, WIDE, LANES>(p, token, lane, nan);
    else expert = choose<PER, WIDE, FP32, LANES>(p, token, lane, nan);
    const float chosen = expert >= 0 ? load_logit(p.logits, FP32, token * p.E + expert) : -__builtin_inff();
    const float top = lanes_max<LANES>(chosen);
    const float mine = expert >= 0 ? expf(chosen - top) : 0.f;
    float sum = mine;
    if (!p.renormalize) {
        float v[PER];
        load_row<PER, WIDE, FP32, LANES>(p.logits, token, p.E, lane, v);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += v[i] > -__builtin_inff() ? expf(v[i] - top) : 0.f;
    }
    sum = lanes_sum<LANES>(sum);
    weight = expert >= 0 ? mine / sum : 0.f;
    if (lanes_reduce<LANES>(nan, [](uint32_t a, uint32_t b) { return a | b; })) weight = __builtin_nanf("");
}

// How a kernel chooses: by sixteen lanes (PER of 16 PER >= E), or by waves (PER of 64 PER >= E).
template <int PER_, bool WIDE_, bool FP32_, bool WAVE_>
struct Choice {
    static constexpr int PER = PER_, experts = (WAVE_ ? 64 : 16) * PER_;
    static constexpr bool WIDE = WIDE_, FP32 = FP32_, WAVE = WAVE_;
};

// The chosen experts and weights of up to 64 tokens, and their masks.
template <typename C>
__device__ __forceinline__ void select_block(const RouteArgs& p, unsigned long long* mask, int64_t first, int count) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
    constexpr int LANES = C::WAVE ? 64 : 16;
    const int lane = threadIdx.x % LANES;
    for (int t = threadIdx.x / LANES; t < count; t += 64 * kRouteWaves / LANES) {
        int expert;
        float weight;
        select<C::PER, C::WIDE, C::FP32, LANES>(p, first + t, lane, expert, weight);
        if (lane < p.top_k) {
            const int64_t at = (first + t) * p.top_k + lane;
            p.experts[at] = expert;
            p.weights[at] = weight;
            if (expert >= 0) atomicOr(mask + expert, 1ull << t);
        }
    }
    __syncthreads();
}

// Exclusive prefix sums of counts(e) over the experts into start[], by the whole workgroup; returns their sum.
template <typename F>
__device__ __forceinline__ int expert_starts(int E, int* start, int* scratch, F counts) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int mine = tid < E ? counts(tid) : 0;                // (E <= 1024 threads)
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        if (lane >= d) sum += v;
    }
    if (lane == 63) scratch[wave] = sum;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        if (w < wave) before += scratch[w];
        total += scratch[w];
    }
    if (tid < E) start[tid] = before + sum - mine;
    __syncthreads();
    return total;
}

// The pairs of up to 64 tokens at their rows: start[e] + rank.  Without an expert no row, and a mark that the combination
// passes on where the token's weights are NaN: logits that are all NaN would else look like padding there.
__device__ __forceinline__ void place_block(const RouteArgs& p, const unsigned long long* mask, const int* start,
                                            int64_t first, int count) {
    for (int s = threadIdx.x; s < count * p.top_k; s += blockDim.x) {
        const int64_t at = first * p.top_k + s;
        const int t = s / p.top_k, e = p.experts[at];
        int row = -1;
        if (e >= 0) {
            row = start[e] + __popcll(mask[e] & ((1ull << t) - 1));
            p.tokens[row] = static_cast<int>(first) + t;
        } else if (p.weights[at] != p.weights[at]) {
            row = EXPERTS_NAN_ROW;
        }
        p.positions[at] = row;
    }
}

// All of it in one workgroup.
template <typename C>
__global__ __launch_bounds__(64 * kRouteWaves) void route_small_kernel(const RouteArgs p) {
    __shared__ unsigned long long mask[C::experts];
    __shared__ int start[C::experts], scratch[kRouteWaves];
    const int count = static_cast<int>(p.T);
    select_block<C>(p, mask, 0, count);
    const int total = expert_starts(p.E, start, scratch, [&](int e) { return __popcll(mask[e]); });
    if (static_cast<int>(threadIdx.x) < p.E) p.offsets[threadIdx.x] = start[threadIdx.x];
    if (threadIdx.x == 0) p.offsets[p.E] = total;
    place_block(p, mask, start, 0, count);
    for (int64_t r = total + threadIdx.x; r < p.T * p.top_k; r += blockDim.x) p.tokens[r] = -1;
}

// Else three launches: choice and counts of every 64 tokens, the counts' sums over the blocks, the placing.
template <typename C>
__global__ __launch_bounds__(64 * kRouteWaves) void route_select_kernel(const RouteArgs p) {
    __shared__ unsigned long long mask[C::experts];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kTokens;
    const int count = static_cast<int>(min(static_cast<int64_t>(kTokens), p.T - first));
    select_block<C>(p, mask, first, count);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
        p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = __popcll(mask[e]);
}

// Sixteen experts a workgroup (neighbours in a line of counts), 64 runs of blocks each; a wave sums up an expert's runs.
constexpr int kScanExperts = 16, kScanRuns = 64;
__global__ __launch_bounds__(kScanExperts * kScanRuns) void route_scan_kernel(const RouteArgs p) {
    __shared__ int sums[kScanRuns][kScanExperts + 1];
    const int x = threadIdx.x % kScanExperts, run = threadIdx.x / kScanExperts, e = blockIdx.x * kScanExperts + x;
    const int per = (p.blocks + kScanRuns - 1) / kScanRuns;
    const int begin = min(run * per, p.blocks), end = e < p.E ? min(begin + per, p.blocks) : begin;
    int* counts = p.counts + e;
    int mine = 0;
#pragma unroll 8
    for (int b = begin; b < end; ++b) mine += counts[static_cast<int64_t>(b) * p.E];
    sums[run][x] = mine;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int value = sums[lane][wave];
    int sum = value;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d, 64);
        if (lane >= d) sum += v;
    }
    sums[lane][wave] = sum - value;
    if (lane == 63 && blockIdx.x * kScanExperts + wave < p.E) p.totals[blockIdx.x * kScanExperts + wave] = sum;
    __syncthreads();
    int before = sums[run][x];
#pragma unroll 8
    for (int b = begin; b < end; ++b) {
        int* at = counts + static_cast<int64_t>(b) * p.E;
        const int c = *at;
        *at = before;
        before += c;
    }
}

__global__ __launch_bounds__(64 * kRouteWaves) void route_place_kernel(const RouteArgs p) {
    __shared__ unsigned long long mask[kMaxExperts];
    __shared__ int start[kMaxExperts], scratch[kRouteWaves];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kTokens;
    const int count = static_cast<int>(min(static_cast<int64_t>(kTokens), p.T - first));
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    const int total = expert_starts(p.E, start, scratch, [&](int e) { return p.totals[e]; });
    if (blockIdx.x == 0) {
        if (static_cast<int>(threadIdx.x) < p.E) p.offsets[threadIdx.x] = start[threadIdx.x];
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    for (int s = threadIdx.x; s < count * p.top_k; s += blockDim.x) {
        const int e = p.experts[first * p.top_k + s];
        if (e >= 0) atomicOr(mask + e, 1ull << (s / p.top_k));
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.E)
        start[threadIdx.x] += p.counts[static_cast<int64_t>(blockIdx.x) * p.E + threadIdx.x];
    __syncthreads();
    place_block(p, mask, start, first, count);
    const int64_t rows = p.T * p.top_k, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t r = total + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; r < rows; r += step)
        p.tokens[r] = -1;
}

// Sixteen lanes per token.  What belongs to the chosen experts, slot by slot on the lanes, goes to their columns
// through a row in LDS: the finished gradients where the softmax is over them alone, else those of the weights.
template <int PER, bool WIDE, bool FP32>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits, const int* __restrict__ experts,
                                                             const float* __restrict__ dweights, void* __restrict__ dlogits,
                                                             int64_t T, int E, int top_k, bool renormalize) {
    constexpr int PITCH = 16 * PER + 4;
    __shared__ __attribute__((aligned(16))) float rows[16 * PITCH];
    const int lane16 = threadIdx.x & 15;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    float* row = rows + (threadIdx.x >> 4) * PITCH;
    if (token >= T) return;                                    // (sixteen lanes together, and no barrier follows)
    float v[PER];
    load_row<PER, WIDE, FP32>(logits, token, E, lane16, v);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        nan |= v[i] != v[i];
        row[expert_of<PER, WIDE, FP32>(lane16, i)] = 0.f;
    }
    const bool any_nan = row_reduce(nan, [](uint32_t a, uint32_t b) { return a | b; }) != 0;
    // this lane's slots: their experts' logits, in rounds of sixteen
    auto for_slots = [&](auto body) {
        for (int j = lane16; j < top_k; j += 16) {
            const int e = experts[token * top_k + j];
            if (e < 0 || e >= E) continue;
            const float l = load_logit(logits, FP32, token * E + e);
            if (l > -__builtin_inff()) body(e, l, dweights[token * top_k + j]);
        }
    };
    wave_lds_fence();
    float top = -__builtin_inff(), sum = 0.f, c = 0.f;
    if (renormalize) {
        for_slots([&](int, float l, float) { top = fmaxf(top, l); });
        top = lanes_max<16>(top);
        for_slots([&](int, float l, float) { sum += expf(l - top); });
        sum = lanes_sum<16>(sum);
        for_slots([&](int, float l, float dw) { c += expf(l - top) / sum * dw; });
        c = lanes_sum<16>(c);
        for_slots([&](int e, float l, float dw) { row[e] = expf(l - top) / sum * (dw - c); });
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = row[expert_of<PER, WIDE, FP32>(lane16, i)];
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) top = fmaxf(top, v[i]);
        top = lanes_max<16>(top);
        for_slots([&](int e, float, float dw) { row[e] = dw; });
        // (masked experts, marked by -1, take no part; beside an infinite logit the sum is NaN, for all others)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = v[i] > -__builtin_inff();
            const float e = in ? expf(v[i] - top) : 0.f;
            sum += e;
            v[i] = in ? e : -1.f;
        }
        sum = lanes_sum<16>(sum);
        for_slots([&](int, float l, float dw) { c += expf(l - top) / sum * dw; });
        c = lanes_sum<16>(c);
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = v[i] == -1.f ? 0.f : v[i] / sum * (row[expert_of<PER, WIDE, FP32>(lane16, i)] - c);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = any_nan ? __builtin_nanf("") : v[i];
    if constexpr (WIDE) {
        constexpr int WORDS = PER * (FP32 ? 4 : 2) / 4;
        uint32_t* out = static_cast<uint32_t*>(dlogits) + token * 16 * WORDS;
        uint32_t w[WORDS];
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            w[i] = FP32 ? __float_as_uint(v[i * PER / WORDS]) : pack_bf16(v[2 * i % PER], v[(2 * i + 1) % PER]);
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4)
                *reinterpret_cast<u32x4_t*>(out + 4 * lane16 + 16 * i) = u32x4_t{w[i], w[i + 1], w[i + 2], w[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) out[lane16 * WORDS + i] = w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<PER, false, FP32>(lane16, i);
            if (e >= E) continue;
            if (FP32)
                static_cast<float*>(dlogits)[token * E + e] = v[i];
            else
                static_cast<uint16_t*>(dlogits)[token * E + e] = f32_to_bf16_bits(v[i]);
        }
    }
}

// Eight columns a thread, in fp32, the experts in their order.  WIDE: rows of whole 16 bytes.  Bound by memory: rows
// are met once, so they are read streamed, four or eight on their way in a thread (8191 tokens of 2560 values, eight
// rows each, 377 MB: 64 us, 5.9 TB/s; with ordinary loads 94).
template <bool WIDE, int HELD>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y, const int* __restrict__ positions,
                                                      const float* __restrict__ weights, uint16_t* __restrict__ out,
                                                      int64_t T, int top_k, int64_t R, int N, int pieces) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t token = at / pieces;
    const int n = 8 * static_cast<int>(at - token * pieces);
    if (token >= T) return;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    float lost = 0.f;                      // (a sum is never -0: adding this one leaves its bits)
    // HELD rows on their way at a time
    for (int j0 = 0; j0 < top_k; j0 += HELD) {
        int64_t row[HELD];
        float w[HELD];
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int64_t slot = token * top_k + min(j0 + j, top_k - 1);
            row[j] = positions[slot];
            w[j] = weights ? weights[slot] : 1.f;
            if (row[j] == EXPERTS_NAN_ROW) lost = __builtin_nanf("");
            if (j0 + j >= top_k || row[j] >= R) row[j] = -1;
        }
        if constexpr (WIDE) {
            u32x4_t v[HELD];
#pragma unroll
            for (int j = 0; j < HELD; ++j)
                v[j] = row[j] < 0 ? u32x4_t{0, 0, 0, 0}
                                  : __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(y + row[j] * N + n));
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                if (row[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[2 * i] += w[j] * __uint_as_float(v[j][i] << 16);
                    sum[2 * i + 1] += w[j] * __uint_as_float(v[j][i] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                if (row[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (n + i < N) sum[i] += w[j] * bf16_bits_to_f32(y[row[j] * N + n + i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += lost;
    uint16_t* to = out + token * N + n;
    if constexpr (WIDE) {
        *reinterpret_cast<u32x4_t*>(to) = u32x4_t{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]),
                                                  pack_bf16(sum[4], sum[5]), pack_bf16(sum[6], sum[7])};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N) to[i] = f32_to_bf16_bits(sum[i]);
    }
}

// A wave per pair of a token and an expert, so that no sum leaves a wave and dout's row comes from the caches for all but
// the first pair of a token.  Bound by memory: the same sizes, 713 MB, take 127 us, 5.6 TB/s (ordinary loads and
// stores, one piece at a time, 133 to 147).
template <bool WIDE>
__global__ __launch_bounds__(256) void combine_backward_kernel(const uint16_t* __restrict__ dout,
                                                               const uint16_t* __restrict__ y,
                                                               const int* __restrict__ positions,
                                                               const float* __restrict__ weights, uint16_t* __restrict__ dy,
                                                               float* __restrict__ dweights, int64_t slots, int top_k,
                                                               int64_t R, int N) {
    const int lane = threadIdx.x & 63;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (slot >= slots) return;
    const int64_t row = positions[slot], token = slot / top_k;
    if (row < 0 || row >= R) {
        if (lane == 0) dweights[slot] = row == EXPERTS_NAN_ROW ? __builtin_nanf("") : 0.f;
        return;
    }
    const float w = weights[slot];
    const uint16_t *d = dout + token * N, *in = y + row * N;
    uint16_t* to = dy + row * N;
    float dot = 0.f;
    if constexpr (WIDE) {
        // five pieces of both rows on their way at a time
        constexpr int HELD = 5;
        for (int n0 = 8 * lane; n0 < N; n0 += 512 * HELD) {
            u32x4_t a[HELD], b[HELD];
#pragma unroll
            for (int q = 0; q < HELD; ++q) {
                const int n = n0 + 512 * q;
                b[q] = n < N ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(in + n)) : u32x4_t{0, 0, 0, 0};
                a[q] = n < N ? load16(d + n) : u32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int q = 0; q < HELD; ++q) {
                const int n = n0 + 512 * q;
                u32x4_t r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = __uint_as_float(a[q][i] << 16), a1 = __uint_as_float(a[q][i] & 0xFFFF0000u);
                    dot += a0 * __uint_as_float(b[q][i] << 16) + a1 * __uint_as_float(b[q][i] & 0xFFFF0000u);
                    r[i] = pack_bf16(w * a0, w * a1);
                }
                if (n < N) __builtin_nontemporal_store(r, reinterpret_cast<u32x4_t*>(to + n));
            }
        }
    } else {
        for (int n = lane; n < N; n += 64) {
            const float a = bf16_bits_to_f32(d[n]);
            dot += a * bf16_bits_to_f32(in[n]);
            to[n] = f32_to_bf16_bits(w * a);
        }
    }
    dot = wave_sum(dot);
    if (lane == 0) dweights[slot] = dot;
}

// body(a Choice by sixteen lanes) for E experts; rows of logits at `base` (and `other`).
template <typename F>
hipError_t for_experts(int E, bool fp32, const void* base, const void* other, F body) {
    auto types = [&](auto per) {
        constexpr int PER = decltype(per)::value;
        const uintptr_t where = reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(other);
        const bool wide = E == 16 * PER && (where & (fp32 ? (PER >= 4 ? 15 : 3) : (PER >= 8 ? 15 : 3))) == 0;
        if (fp32) return wide ? body(Choice<PER, true, true, false>{}) : body(Choice<PER, false, true, false>{});
        if constexpr (PER >= 2)
            if (wide) return body(Choice<PER, true, false, false>{});
        return body(Choice<PER, false, false, false>{});
    };
    if (E <= 16) return types(std::integral_constant<int, 1>{});
    if (E <= 32) return types(std::integral_constant<int, 2>{});
    if (E <= 64) return types(std::integral_constant<int, 4>{});
    if (E <= 128) return types(std::integral_constant<int, 8>{});
    if (E <= 256) return types(std::integral_constant<int, 16>{});
    if (E <= 512) return types(std::integral_constant<int, 32>{});
    return types(std::integral_constant<int, 64>{});
}

}  // namespace

uint64_t experts_route_bytes(int64_t T, int E) {
    if (T <= kTokens) return 0;
    return static_cast<uint64_t>((T + kTokens - 1) / kTokens + 1) * E * sizeof(int);
}

hipError_t launch_experts_route(const void* logits, bool fp32, int top_k, bool renormalize, float* weights, int* experts,
                                int* positions, int* tokens, int* offsets, int64_t T, int E, int* ws, hipStream_t stream) {
    const int blocks = static_cast<int>((T + kTokens - 1) / kTokens);
    const RouteArgs args{logits, weights, experts, positions, tokens, offsets, ws, ws ? ws + static_cast<int64_t>(blocks) * E : nullptr,
                         T, E, top_k, blocks, fp32, renormalize};
    const dim3 threads(64 * kRouteWaves);
    auto run = [&](auto choice) {
        using C = decltype(choice);
        if (T <= kTokens) {
            hipLaunchKernelGGL(route_small_kernel<C>, dim3(1), threads, 0, stream, args);
            return hipGetLastError();
        }
        hipLaunchKernelGGL(route_select_kernel<C>, dim3(blocks), threads, 0, stream, args);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(route_scan_kernel, dim3((E + kScanExperts - 1) / kScanExperts), dim3(kScanExperts * kScanRuns), 0,
                           stream, args);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(route_place_kernel, dim3(blocks), threads, 0, stream, args);
        return hipGetLastError();
    };
    // A wave a token for more than sixteen chosen experts, and where sixteen lanes would have 64 logits each, unless they
    // are whole rows of bf16 (32768 x 1024, eight chosen: fp32 70 us, by sixteen lanes 128; bf16 80 and 52; x 1000 79 and 93).
    auto by_waves = [&](auto types) {
        constexpr bool F = decltype(types)::value;
        if (E <= 128) return run(Choice<2, false, F, true>{});
        return E <= 512 ? run(Choice<8, false, F, true>{}) : run(Choice<16, false, F, true>{});
    };
    if (top_k > 16) return fp32 ? by_waves(std::true_type{}) : by_waves(std::false_type{});
    return for_experts(E, fp32, logits, nullptr, [&](auto choice) {
        using C = decltype(choice);
        if constexpr (C::PER == 64 && (C::FP32 || !C::WIDE)) return run(Choice<16, false, C::FP32, true>{});
        else return run(choice);
    });
}

hipError_t launch_experts_route_backward(const void* logits, bool fp32, const int* experts, const float* dweights,
                                         void* dlogits, int64_t T, int E, int top_k, bool renormalize,
                                         hipStream_t stream) {
    return for_experts(E, fp32, logits, dlogits, [&](auto choice) {
        using C = decltype(choice);
        hipLaunchKernelGGL((route_backward_kernel<C::PER, C::WIDE, C::FP32>), dim3(static_cast<uint32_t>((T + 15) / 16)), dim3(256), 0,
                           stream, logits, experts, dweights, dlogits, T, E, top_k, renormalize);
        return hipGetLastError();
    });
}

hipError_t launch_experts_combine(const uint16_t* y, const int* positions, const float* weights, uint16_t* out, int64_t T,
                                  int top_k, int64_t R, int N, hipStream_t stream) {
    const int pieces = (N + 7) / 8;
    const dim3 grid(static_cast<uint32_t>((T * pieces + 255) / 256)), threads(256);
    const bool wide = N % 8 == 0 && ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, threads, 0, stream, y, positions, weights, out, T, top_k, R, N, pieces);
    };
    if (!wide) run(combine_kernel<false, 4>);
    else if (top_k <= 2) run(combine_kernel<true, 2>);
    else if (top_k <= 4) run(combine_kernel<true, 4>);
    else run(combine_kernel<true, 8>);
    return hipGetLastError();
}

hipError_t launch_experts_combine_backward(const uint16_t* dout, const uint16_t* y, const int* positions,
                                           const float* weights, uint16_t* dy, float* dweights, int64_t T, int top_k,
                                           int64_t R, int N, hipStream_t stream) {
    const int64_t slots = T * top_k;
    const dim3 grid(static_cast<uint32_t>((slots + 3) / 4)), threads(256);
    const bool wide = N % 8 == 0 && ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(dout) |
                                      reinterpret_cast<uintptr_t>(dy)) & 15) == 0;
    if (wide)
        hipLaunchKernelGGL(combine_backward_kernel<true>, grid, threads, 0, stream, dout, y, positions, weights, dy, dweights,
                           slots, top_k, R, N);
    else
        hipLaunchKernelGGL(combine_backward_kernel<false>, grid, threads, 0, stream, dout, y, positions, weights, dy, dweights,
                           slots, top_k, R, N);
    return hipGetLastError();
}

}  // namespace w4a16
