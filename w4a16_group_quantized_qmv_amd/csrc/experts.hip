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
// Bound by latency up to some hundred tokens (one launch of one workgroup), by reading and writing once above.
#include "device_common.h"
#include "mxfp4_device.h"
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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
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

// One token by one wave: lane j < top_k gets the j-th chosen expert (-1 for none) and its weight.  PER logits a
// lane, expert lane + 64 i.
template <int PER>
__device__ __forceinline__ void select(const RouteArgs& p, int64_t token, int lane, int& expert, float& weight) {
    float v[PER];
    uint32_t key[PER];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < p.E ? load_logit(p.logits, p.fp32, token * p.E + e) : -__builtin_inff();
        nan |= v[i] != v[i];
        key[i] = order_key(v[i]);
    }
    expert = -1;
    float chosen = 0.f, top = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        // the larger key wins, of equal ones the lower expert
        uint64_t pair = (static_cast<uint64_t>(best) << 32) | static_cast<uint32_t>(0xFFFF - (lane + 64 * at));
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            const uint64_t other = __shfl_xor(pair, d, 64);
            pair = other > pair ? other : pair;
        }
        const uint32_t won = static_cast<uint32_t>(pair >> 32);
        if (won == 0) break;                                   // (uniform) nothing is left
        const int e = 0xFFFF - static_cast<int>(static_cast<uint32_t>(pair));
        const float logit = __uint_as_float((won >> 31) ? won & 0x7FFFFFFFu : ~won);
        if (j == 0) top = logit;
        if (lane == j) {
            expert = e;
            chosen = logit;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i == e) key[i] = 0;
    }
    const float mine = expert >= 0 ? expf(chosen - top) : 0.f;
    float sum = 0.f;
    if (p.renormalize) {
        sum = wave_sum(mine);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += v[i] > -__builtin_inff() ? expf(v[i] - top) : 0.f;
        sum = wave_sum(sum);
    }
    weight = expert >= 0 ? mine / sum : 0.f;
    if (__ballot(nan)) weight = __builtin_nanf("");
}

// The chosen experts and weights of up to 64 tokens, and their masks.
template <int PER>
__device__ __forceinline__ void select_block(const RouteArgs& p, unsigned long long* mask, int64_t first, int count) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
    for (int t = wave; t < count; t += kRouteWaves) {
        int expert;
        float weight;
        select<PER>(p, first + t, lane, expert, weight);
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

// The pairs of up to 64 tokens at their rows: start[e] + rank.
__device__ __forceinline__ void place_block(const RouteArgs& p, const unsigned long long* mask, const int* start,
                                            int64_t first, int count) {
    for (int s = threadIdx.x; s < count * p.top_k; s += blockDim.x) {
        const int64_t at = first * p.top_k + s;
        const int t = s / p.top_k, e = p.experts[at];
        int row = -1;
        if (e >= 0) {
            row = start[e] + __popcll(mask[e] & ((1ull << t) - 1));
            p.tokens[row] = static_cast<int>(first) + t;
        }
        p.positions[at] = row;
    }
}

// All of it in one workgroup.
template <int PER>
__global__ __launch_bounds__(64 * kRouteWaves) void route_small_kernel(const RouteArgs p) {
    __shared__ unsigned long long mask[64 * PER];
    __shared__ int start[64 * PER], scratch[kRouteWaves];
    const int count = static_cast<int>(p.T);
    select_block<PER>(p, mask, 0, count);
    const int total = expert_starts(p.E, start, scratch, [&](int e) { return __popcll(mask[e]); });
    if (static_cast<int>(threadIdx.x) < p.E) p.offsets[threadIdx.x] = start[threadIdx.x];
    if (threadIdx.x == 0) p.offsets[p.E] = total;
    place_block(p, mask, start, 0, count);
    for (int64_t r = total + threadIdx.x; r < p.T * p.top_k; r += blockDim.x) p.tokens[r] = -1;
}

// Else three launches: choice and counts of every 64 tokens, the counts' sums over the blocks, the placing.
template <int PER>
__global__ __launch_bounds__(64 * kRouteWaves) void route_select_kernel(const RouteArgs p) {
    __shared__ unsigned long long mask[64 * PER];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kTokens;
    const int count = static_cast<int>(min(static_cast<int64_t>(kTokens), p.T - first));
    select_block<PER>(p, mask, first, count);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
        p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = __popcll(mask[e]);
}

// Sixteen experts a workgroup, 64 runs of blocks each.
constexpr int kScanExperts = 16, kScanRuns = 64;
__global__ __launch_bounds__(kScanExperts * kScanRuns) void route_scan_kernel(const RouteArgs p) {
    __shared__ int sums[kScanRuns][kScanExperts + 1];
    const int x = threadIdx.x % kScanExperts, run = threadIdx.x / kScanExperts;
    const int e = blockIdx.x * kScanExperts + x;
    const int per = (p.blocks + kScanRuns - 1) / kScanRuns;
    const int begin = min(run * per, p.blocks), end = min(begin + per, p.blocks);
    int sum = 0;
    if (e < p.E)
        for (int b = begin; b < end; ++b) sum += p.counts[static_cast<int64_t>(b) * p.E + e];
    sums[run][x] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int r = 0; r < kScanRuns; ++r) {
        if (r < run) before += sums[r][x];
        total += sums[r][x];
    }
    if (e >= p.E) return;
    for (int b = begin; b < end; ++b) {
        int* at = p.counts + static_cast<int64_t>(b) * p.E + e;
        const int c = *at;
        *at = before;
        before += c;
    }
    if (run == 0) p.totals[e] = total;
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

// A wave per token.  The gradients of the chosen experts go to their columns through a row in LDS.
template <int PER>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits, bool fp32,
                                                             const int* __restrict__ experts,
                                                             const float* __restrict__ dweights, void* __restrict__ dlogits,
                                                             int64_t T, int E, int top_k, bool renormalize) {
    __shared__ float row[4][64 * PER];
    __shared__ uint8_t picked[4][64 * PER];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * 4 + wave;
    if (token >= T) return;
    float v[PER];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? load_logit(logits, fp32, token * E + e) : -__builtin_inff();
        nan |= v[i] != v[i];
        row[wave][e] = 0.f;
        picked[wave][e] = 0;
    }
    wave_lds_fence();
    if (lane < top_k) {
        const int e = experts[token * top_k + lane];
        if (e >= 0 && e < E) {
            row[wave][e] = dweights[token * top_k + lane];
            picked[wave][e] = 1;
        }
    }
    wave_lds_fence();
    const bool any_nan = __ballot(nan) != 0;
    float top = -__builtin_inff();
    bool in[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        in[i] = v[i] > -__builtin_inff() && (!renormalize || picked[wave][lane + 64 * i]);
        if (in[i]) top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    float p[PER], sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        p[i] = in[i] ? expf(v[i] - top) : 0.f;
        sum += p[i];
    }
    sum = wave_sum(sum);
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        p[i] = in[i] ? p[i] / sum : 0.f;
        if (in[i]) c += p[i] * row[wave][lane + 64 * i];
    }
    c = wave_sum(c);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        float d = in[i] ? p[i] * (row[wave][e] - c) : 0.f;
        if (any_nan) d = __builtin_nanf("");
        if (fp32)
            static_cast<float*>(dlogits)[token * E + e] = d;
        else
            static_cast<uint16_t*>(dlogits)[token * E + e] = f32_to_bf16_bits(d);
    }
}

// Eight columns a thread, in fp32, the experts in their order.  WIDE: rows of whole 16 bytes.
template <bool WIDE>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y, const int* __restrict__ positions,
                                                      const float* __restrict__ weights, uint16_t* __restrict__ out,
                                                      int64_t T, int top_k, int64_t R, int N, int pieces) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t token = at / pieces;
    const int n = 8 * static_cast<int>(at - token * pieces);
    if (token >= T) return;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j = 0; j < top_k; ++j) {
        const int64_t row = positions[token * top_k + j];
        if (row < 0 || row >= R) continue;
        const float w = weights ? weights[token * top_k + j] : 1.f;
        const uint16_t* in = y + row * N + n;
        if constexpr (WIDE) {
            const u32x4_t v = load16(in);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[2 * i] += w * __uint_as_float(v[i] << 16);
                sum[2 * i + 1] += w * __uint_as_float(v[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n + i < N) sum[i] += w * bf16_bits_to_f32(in[i]);
        }
    }
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

// A wave per pair of a token and an expert.
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
        if (lane == 0) dweights[slot] = 0.f;
        return;
    }
    const float w = weights[slot];
    const uint16_t *d = dout + token * N, *in = y + row * N;
    uint16_t* to = dy + row * N;
    float dot = 0.f;
    if constexpr (WIDE) {
        for (int n = 8 * lane; n < N; n += 512) {
            const u32x4_t a = load16(d + n), b = load16(in + n);
            u32x4_t r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = __uint_as_float(a[i] << 16), a1 = __uint_as_float(a[i] & 0xFFFF0000u);
                dot += a0 * __uint_as_float(b[i] << 16) + a1 * __uint_as_float(b[i] & 0xFFFF0000u);
                r[i] = pack_bf16(w * a0, w * a1);
            }
            *reinterpret_cast<u32x4_t*>(to + n) = r;
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

// body(std::integral_constant<int, logits of a lane>).
template <typename F>
hipError_t for_experts(int E, F body) {
    if (E <= 64) return body(std::integral_constant<int, 1>{});
    if (E <= 128) return body(std::integral_constant<int, 2>{});
    if (E <= 256) return body(std::integral_constant<int, 4>{});
    if (E <= 512) return body(std::integral_constant<int, 8>{});
    return body(std::integral_constant<int, 16>{});
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
    return for_experts(E, [&](auto per) {
        constexpr int PER = decltype(per)::value;
        if (T <= kTokens) {
            hipLaunchKernelGGL(route_small_kernel<PER>, dim3(1), threads, 0, stream, args);
            return hipGetLastError();
        }
        hipLaunchKernelGGL(route_select_kernel<PER>, dim3(blocks), threads, 0, stream, args);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(route_scan_kernel, dim3((E + kScanExperts - 1) / kScanExperts), dim3(kScanExperts * kScanRuns), 0,
                           stream, args);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(route_place_kernel, dim3(blocks), threads, 0, stream, args);
        return hipGetLastError();
    });
}

hipError_t launch_experts_route_backward(const void* logits, bool fp32, const int* experts, const float* dweights,
                                         void* dlogits, int64_t T, int E, int top_k, bool renormalize,
                                         hipStream_t stream) {
    return for_experts(E, [&](auto per) {
        hipLaunchKernelGGL(route_backward_kernel<decltype(per)::value>, dim3(static_cast<uint32_t>((T + 3) / 4)), dim3(256), 0,
                           stream, logits, fp32, experts, dweights, dlogits, T, E, top_k, renormalize);
        return hipGetLastError();
    });
}

hipError_t launch_experts_combine(const uint16_t* y, const int* positions, const float* weights, uint16_t* out, int64_t T,
                                  int top_k, int64_t R, int N, hipStream_t stream) {
    const int pieces = (N + 7) / 8;
    const dim3 grid(static_cast<uint32_t>((T * pieces + 255) / 256)), threads(256);
    const bool wide = N % 8 == 0 && ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    if (wide)
        hipLaunchKernelGGL(combine_kernel<true>, grid, threads, 0, stream, y, positions, weights, out, T, top_k, R, N, pieces);
    else
        hipLaunchKernelGGL(combine_kernel<false>, grid, threads, 0, stream, y, positions, weights, out, T, top_k, R, N, pieces);
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
