// experts.hpp -- gfx950 kernels of the mixture-of-experts calls: top-k
// routing of router logits, the stable sort of (token, choice) slots by
// expert, and the movement of token rows to their sorted places and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "device.hpp"
#include "elements.hpp"

namespace rs {

// The sum of f(x of lane b) over the other lanes b of a group of G: the group's
// rows of 16 lanes take turns, each rotated past the lane (DPP row_ror).
template <int BY>
__device__ __forceinline__ uint32_t rotated(uint32_t x) {
    return dpp<0x120 + BY>(x);
}
template <int BY>
__device__ __forceinline__ uint64_t rotated(uint64_t x) {
    return static_cast<uint64_t>(dpp<0x120 + BY>(static_cast<uint32_t>(x >> 32))) << 32 |
           dpp<0x120 + BY>(static_cast<uint32_t>(x));
}
template <class U, class F, int... I>
__device__ __forceinline__ int sum_rotated(const U &x, F &&f, std::integer_sequence<int, I...>) {
    return (f(rotated<I + 1>(x)) + ...);
}
template <int G, class U, class F>
__device__ __forceinline__ int sum_over_others(const U &x, F &&f) {
    int sum = sum_rotated(x, f, std::make_integer_sequence<int, 15>{});
#pragma unroll
    for (int row = 16; row < G; row += 16) {
        const U other = __shfl_xor(x, row);
        sum += f(other) + sum_rotated(other, f, std::make_integer_sequence<int, 15>{});
    }
    return sum;
}

// The sum of x up to each lane of its group of G.
template <int G>
__device__ __forceinline__ uint32_t group_inclusive_sum(uint32_t x) {
    if constexpr (G == 64) return wave_inclusive_sum(x);
    const auto below = [](uint32_t y, auto ctrl, auto rows) {
        return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(y), decltype(ctrl)::value,
                                                                 decltype(rows)::value, 0xF, false));
    };
    using All = std::integral_constant<int, 0xF>;
    x += below(x, std::integral_constant<int, 0x111>{}, All{});  // row_shr 1, 2, 4, 8
    x += below(x, std::integral_constant<int, 0x112>{}, All{});
    x += below(x, std::integral_constant<int, 0x114>{}, All{});
    x += below(x, std::integral_constant<int, 0x118>{}, All{});
    if constexpr (G == 32) {  // row_bcast15 into rows 1 and 3
        x += below(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
    }
    return x;
}

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
constexpr int kRouteBlock = 256;

// Rank of a logit as an unsigned integer: a larger logit has a larger rank,
// -0 equals +0, every NaN ranks above every number, and -inf (an expert that
// the row may not use) has rank 0, below every finite value.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t bits = __float_as_uint(x + 0.0f);
    if (x == -__builtin_inff()) return 0;
    if (x != x) return 0xFFFFFFFFu;
    return (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
}

__device__ __forceinline__ float ranked_value(uint32_t rank) {
    return __uint_as_float((rank & 0x80000000u) ? (rank ^ 0x80000000u) : ~rank);
}

enum : int { kGateSoftmax = 0, kGateSigmoid = 1 };

// 1 / (1 + exp(-l)), and its complement as sigmoid(-l); exp only of numbers
// <= 0, so neither end overflows.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-__builtin_fabsf(l));
    return (l >= 0.0f || l != l ? 1.0f : e) / (1.0f + e);
}

// exp(t) for t <= 0 as a share of a sum that holds a 1: exp2 of t * log2(e) in
// two parts, without the range steps of expf (a result below 2^-126 may be 0).
__device__ __forceinline__ float exp_in_sum(float t) {
    constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147182f;
    t = t < -200.0f ? -200.0f : t;  // keeps the parts finite (a NaN stays one)
    const float hi = t * kLog2e;
    const float lo = __builtin_fmaf(t, kLog2eRest, __builtin_fmaf(t, kLog2e, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(e, lo * kLn2, e);
}

// A row's logits in G lanes, V each: lane g holds the elements
// (c * G + g) * W + w of chunk c.
template <int G, int V, int W>
__device__ __forceinline__ int held_index(int g, int v) {
    return ((v / W) * G + g) * W + v % W;
}

// Loads a row so; -inf beyond its end.  No load waits for a branch: lanes beyond
// the end read its last elements again, and a row whose length is no multiple
// of an access is read by elements.
template <class T, int G, int V, int W>
__device__ __forceinline__ void hold_row(const T *row, int experts, int g, float (&x)[V]) {
    if (experts % W == 0) {
#pragma unroll
        for (int c = 0; c < V / W; ++c) {
            const int i0 = (c * G + g) * W;
            float f[W];
            load_vec<T, W>(row + (i0 < experts ? i0 : experts - W), f);
#pragma unroll
            for (int w = 0; w < W; ++w) x[c * W + w] = i0 < experts ? f[w] : -__builtin_inff();
        }
    } else {
        T f[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = held_index<G, V, W>(g, v);
            f[v] = row[i < experts ? i : experts - 1];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = held_index<G, V, W>(g, v) < experts ? static_cast<float>(f[v]) : -__builtin_inff();
        }
    }
}

// Rounds of taking the group's largest rank, at its lowest index: lane j keeps
// round j's winner (rank 0: none was left), so k <= G.
template <int G, int V, int W>
__device__ __forceinline__ void choose_by_rounds(const float (&x)[V], int g, int k, uint32_t &my_rank,
                                                 uint32_t &my_index) {
    uint32_t rank[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rank[v] = rank_of(x[v]);
    my_rank = my_index = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = rank[0], at = 0xFFFFFFFFu;
#pragma unroll
        for (int v = 1; v < V; ++v) best = rank[v] > best ? rank[v] : best;
        best = group_max_u32<G>(best);
#pragma unroll
        for (int v = V - 1; v >= 0; --v) at = rank[v] == best ? static_cast<uint32_t>(held_index<G, V, W>(g, v)) : at;
        at = group_min_u32<G>(at);
#pragma unroll
        for (int v = 0; v < V; ++v) rank[v] = static_cast<uint32_t>(held_index<G, V, W>(g, v)) == at ? 0u : rank[v];
        my_rank = g == j ? best : my_rank;
        my_index = g == j ? at : my_index;
    }
}

// Orders the `total` logits whose indices are in room[0 .. total): N to a lane,
// where each counts the better ones (larger, or equal with a lower index).
// Lane j < k gets the j-th best, if there is one.
template <class T, int G, int N>
__device__ __forceinline__ void place_by_counts(const T *row, int g, int k, int total, uint32_t *room, float &value,
                                                uint32_t &index, bool &taken) {
    uint64_t key[N];  // larger value, then lower index, as one number; 0 for no logit
    int better[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bool holds = g + n * G < total;
        const uint32_t i = holds ? room[g + n * G] : 0u;
        key[n] = holds ? static_cast<uint64_t>(rank_of(static_cast<float>(row[i]))) << 32 | (0xFFFFFFFFu - i) : 0u;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        better[n] = 0;
#pragma unroll
        for (int m = 0; m < N; ++m) {
            const auto above = [&](uint64_t other) { return other > key[n] ? 1 : 0; };
            better[n] += sum_over_others<G>(key[m], above) + (m != n ? above(key[m]) : 0);
        }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (g + n * G < total) room[better[n]] = 0xFFFFFFFFu - static_cast<uint32_t>(key[n]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    taken = g < k && g < total;
    index = taken ? room[g] : 0u;
    value = taken ? static_cast<float>(row[index]) : 0.0f;
    __builtin_amdgcn_wave_barrier();
}

// The k-th largest of the G lanes' maxima is at most the row's k-th largest
// logit.  With k <= G / 2 few logits of a random row of any length reach it, 11
// for k = 8 of 16 lanes (16 * (1/9 + ... + 1/16)), 22 for 16 of 32, 44 for 32 of
// 64: they mostly fit one to a lane.  Rows of 16 lanes, which exceed that the most
// often (1% of them at k = 8), have room for two to a lane; for larger groups
// the registers of a second one would halve the waves in flight (8192 x 1024, k
// = 32: 19.3 us without, 33.6 with).  The lanes pass the indices of theirs
// through `room`.  Returns false, for every lane of the wave, if a row of the
// wave has more such logits (many equal ones, few that are not -inf) or a NaN.
template <class T, int G, int V, int W>
__device__ __forceinline__ bool choose_by_counts(const float (&x)[V], const T *row, int g, int k, uint32_t *room,
                                                 float &value, uint32_t &index, bool &taken) {
    static_assert(V <= 32);
    float most = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) most = __builtin_elementwise_maximum(most, x[v]);
    const int above = sum_over_others<G>(__float_as_uint(most),
                                         [&](uint32_t other) { return __uint_as_float(other) > most ? 1 : 0; });
    constexpr float kInf = __builtin_inff(), kLowest = -3.402823466e38f;
    const float kth = -group_max<G>(above < k ? -most : -kInf);  // NaN with a NaN in the row
    const float least = kth == -kInf ? kLowest : kth;            // -inf is never chosen
    uint32_t mask = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) mask |= x[v] >= least ? 1u << v : 0u;
    const int mine = __popc(mask);
    const int upto = static_cast<int>(group_inclusive_sum<G>(static_cast<uint32_t>(mine)));
    constexpr int kRoom = G == 16 ? 2 * G : G;
    if (__ballot((kth != kth) | (upto > kRoom)) != 0) return false;
    int put = upto - mine;
    for (; mask != 0; mask &= mask - 1) {
        room[put++] = static_cast<uint32_t>(held_index<G, V, W>(g, __ffs(static_cast<int>(mask)) - 1));
    }
    const int total = static_cast<int>(group_max_u32<G>(static_cast<uint32_t>(upto)));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (kRoom == G || __ballot(total > G) == 0) {
        place_by_counts<T, G, 1>(row, g, k, total, room, value, index, taken);
    } else {
        place_by_counts<T, G, kRoom / G>(row, g, k, total, room, value, index, taken);
    }
    return true;
}

// The k largest logits of each row and their weights: a row in G lanes, slot j
// in lane j.  counts: choose_by_counts is tried first (k <= G / 2).
// Each logit is read once; a wave then spends some 390 vector instructions on
// its 64 / G rows, which bounds it together with the one wait for the row.
// 16384 x 256 float32, k = 8: 5.8 us (17.8 MB, 3.1 TB/s) with the rows in the
// last-level cache, 7.3 from memory; in rounds alone 10.1.
template <class T, int G, int V>
__global__ __launch_bounds__(kRouteBlock) void route_topk_kernel(const T *__restrict__ logits, size_t tokens,
                                                                 int experts, size_t stride, int k, int gate,
                                                                 int renormalize, float scale, bool counts,
                                                                 float *__restrict__ weights,
                                                                 int32_t *__restrict__ chosen) {
    constexpr int W = V < kVec<T> ? V : kVec<T>;
    constexpr int kRows = kRouteBlock / G;
    __shared__ uint32_t room[kRows][2 * G];
    const int g = threadIdx.x % G;
    const size_t mine = static_cast<size_t>(blockIdx.x) * kRows + threadIdx.x / G;
    const bool live = mine < tokens;
    const T *row = logits + (live ? mine : tokens - 1) * stride;
    float x[V];
    hold_row<T, G, V, W>(row, experts, g, x);

    float l = 0.0f;
    uint32_t index = 0;
    bool taken = false;
    if (!counts || !choose_by_counts<T, G, V, W>(x, row, g, k, room[threadIdx.x / G], l, index, taken)) {
        uint32_t rank;
        choose_by_rounds<G, V, W>(x, g, k, rank, index);
        taken = g < k && rank != 0;
        l = ranked_value(rank);
    }
    // The largest chosen logit is the row's.
    const float top = group_max<G>(taken ? l : -__builtin_inff());
    float w;
    if (gate == kGateSoftmax) {
        w = taken ? expf(l - top) : 0.0f;
        float total;
        if (renormalize) {
            total = group_sum<G>(w);
        } else {
            total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) total += x[v] == -__builtin_inff() ? 0.0f : exp_in_sum(x[v] - top);
            total = group_sum<G>(total);
        }
        w = w / total;
    } else if (!renormalize) {
        w = sigmoid(l);
    } else {
        // sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)): the common factor
        // exp(min(top, 0)) cancels, so very negative rows keep their ratios.
        const float shift = __builtin_fminf(top, 0.0f);
        const float num = l != l ? l : expf(__builtin_fminf(l, 0.0f) - shift);
        w = taken ? num / (1.0f + expf(-__builtin_fabsf(l))) : 0.0f;
        w = w / group_sum<G>(w);
    }
    if (live && g < k) {
        const size_t at = mine * static_cast<size_t>(k) + g;
        weights[at] = taken ? w * scale : 0.0f;
        chosen[at] = taken ? static_cast<int32_t>(index) : -1;
    }
}

// Gradient of the router logits.  With p the gate's values, u = p / (sum of
// the chosen p), h the incoming gradient and a_i the sum of h over the slots
// that chose i:
//   softmax                dl_i = scale * p_i * (a_i - sum_j h_j p_j)
//   softmax, renormalized  dl_i = scale * u_i * (a_i - sum_j h_j u_j), chosen i only
//   sigmoid                dl_i = scale * a_i * p_i * (1 - p_i), chosen i only
//   sigmoid, renormalized  dl_i = scale * u_i * (a_i - sum_j h_j u_j) * (1 - p_i)
// Only the first needs the whole row; the others read the k chosen logits.  Its
// -0 marks a barred expert, whose gradient is 0 whatever the row holds; an
// exponential that underflows is +0 and follows the formula (a row with a NaN or
// +inf, or a NaN gradient of a weight, has no finite gradient anywhere else).
// Lane j < k of the group holds slot j; the slots' terms reach the lanes that
// hold their elements through LDS.  32768 x 256 float32, softmax, k = 8: 16.1 us
// (69 MB, 4.3 TB/s), not the memory's rate: the choices are loaded after the row
// is summed, then the chosen logits, and two barriers tie four waves together.
template <class T, int G, int V>
__global__ __launch_bounds__(kRouteBlock) void route_topk_backward_kernel(
    const T *__restrict__ logits, size_t tokens, int experts, size_t stride, const int32_t *__restrict__ chosen,
    const float *__restrict__ grad_weights, int k, int gate, int renormalize, float scale,
    T *__restrict__ grad_logits, size_t grad_stride) {
    constexpr int W = V < kVec<T> ? V : kVec<T>;
    constexpr int C = V / W;
    constexpr int kRows = kRouteBlock / G;
    __shared__ float terms[kRows][G * V];
    const int g = threadIdx.x % G;
    const int sub = threadIdx.x / G;
    const bool whole = gate == kGateSoftmax && !renormalize;
    const size_t mine = static_cast<size_t>(blockIdx.x) * kRows + sub;
    const bool live = mine < tokens;
    const size_t r = live ? mine : tokens - 1;
    const T *row = logits + r * stride;

    float p[V];
    float top = 0.0f, total = 1.0f;
    if (whole) {
        hold_row<T, G, V, W>(row, experts, g, p);
        top = p[0];
#pragma unroll
        for (int v = 1; v < V; ++v) top = __builtin_elementwise_maximum(top, p[v]);
        top = group_max<G>(top);
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = p[v] == -__builtin_inff() ? -0.0f : exp_in_sum(p[v] - top);
            total += p[v];
        }
        total = group_sum<G>(total);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int w = 0; w < W; ++w) terms[sub][(c * G + g) * W + w] = 0.0f;
    }

    int32_t s = -1;
    float h = 0.0f, l = -__builtin_inff();
    if (g < k) {
        s = chosen[r * static_cast<size_t>(k) + g];
        if (static_cast<uint32_t>(s) < static_cast<uint32_t>(experts)) {
            l = static_cast<float>(row[s]);
            h = grad_weights[r * static_cast<size_t>(k) + g];
        }
    }
    const bool taken = l != -__builtin_inff();  // a slot without an expert adds nothing
    float d = 0.0f, mean = 0.0f;
    if (whole) {
        mean = group_sum<G>(taken ? h * (expf(l - top) / total) : 0.0f);
        d = h;
    } else if (!renormalize) {
        d = h * sigmoid(l) * sigmoid(-l);
    } else {
        float best = group_max<G>(taken ? l : -__builtin_inff());
        float u;
        if (gate == kGateSoftmax) {
            u = taken ? expf(l - best) : 0.0f;
        } else {
            best = __builtin_fminf(best, 0.0f);
            const float num = l != l ? l : expf(__builtin_fminf(l, 0.0f) - best);
            u = taken ? num / (1.0f + expf(-__builtin_fabsf(l))) : 0.0f;
        }
        u = u / group_sum<G>(u);
        mean = group_sum<G>(taken ? h * u : 0.0f);
        d = u * (h - mean);
        if (gate == kGateSigmoid) d *= sigmoid(-l);
    }
    if (!taken) d = 0.0f;
    // Slots that chose the same expert each store the sum of all of them.
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int sj = __shfl(s, j, G);
        const float dj = __shfl(d, j, G);
        sum += sj == s ? dj : 0.0f;
    }
    __syncthreads();
    if (taken) terms[sub][s] = sum;
    __syncthreads();
    T *out = grad_logits + r * grad_stride;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i0 = (c * G + g) * W;
        float f[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float a = terms[sub][i0 + w];
            if (whole) {
                const float q = p[c * W + w] / total;
                f[w] = __float_as_uint(p[c * W + w]) == 0x80000000u ? 0.0f : scale * (q * (a - mean));
            } else {
                f[w] = scale * a;
            }
        }
        if (live && i0 < experts) store_some<T, W>(out + i0, experts - i0, f);
    }
}

// ---------------------------------------------------------------------------
// Slots sorted by expert
// ---------------------------------------------------------------------------
constexpr int kPlaceBlock = 1024;
constexpr int kPlaceWaves = kPlaceBlock / 64;
constexpr int kMaxExperts = 1024;

// Sort key of a slot: its expert's number among those counted, `experts` for
// an id outside of them (dropped: sorted last).
template <class ID>
__device__ __forceinline__ uint32_t expert_key(ID id, ID first, uint32_t experts) {
    using U = typename std::make_unsigned<ID>::type;
    const U e = static_cast<U>(id) - static_cast<U>(first);
    return e < static_cast<U>(experts) ? static_cast<uint32_t>(e) : experts;
}

// Row length of the count table: whole 16-byte accesses.
constexpr uint32_t table_stride(uint32_t experts) { return (experts + 3u) & ~3u; }

// Experts of each workgroup's chunk of slots, counted in LDS:
// table[workgroup][expert].  One read of the ids: 2.8 us for 2^20 (4 MiB), about
// a launch.
template <class ID, int ITEMS>
__global__ __launch_bounds__(kPlaceBlock) void expert_count_kernel(const ID *__restrict__ ids, size_t n, ID first,
                                                                   uint32_t experts, size_t chunk,
                                                                   uint32_t *__restrict__ table) {
    __shared__ uint32_t count[kMaxExperts + 4];
    const uint32_t stride = table_stride(experts);
    const size_t lo = blockIdx.x * chunk;
    const size_t hi = lo + chunk < n ? lo + chunk : n;
    for (uint32_t e = threadIdx.x; e < stride; e += kPlaceBlock) count[e] = 0;
    __syncthreads();
    for (size_t tile = lo + threadIdx.x; tile < hi; tile += static_cast<size_t>(kPlaceBlock) * ITEMS) {
        ID id[ITEMS];  // all in flight: beyond the chunk the last slot, not counted
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const size_t slot = tile + static_cast<size_t>(i) * kPlaceBlock;
            id[i] = ids[slot < hi ? slot : hi - 1];
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t key = expert_key(id[i], first, experts);
            if (key < experts && tile + static_cast<size_t>(i) * kPlaceBlock < hi) atomicAdd(&count[key], 1u);
        }
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < stride; e += kPlaceBlock) {
        table[static_cast<size_t>(blockIdx.x) * stride + e] = count[e];
    }
}

// Exclusive sums of each expert's column of the table, in place, and the
// columns' totals.  A workgroup takes 64 columns; a thread four of them over
// kScanRows consecutive rows, held in registers.  One round trip to memory,
// about a launch.
constexpr uint32_t kMaxChunks = 256;  // rows of the table
constexpr uint32_t kScanQuads = 16;
constexpr uint32_t kScanSplits = kPlaceBlock / kScanQuads;
constexpr uint32_t kScanRows = kMaxChunks / kScanSplits;

__global__ __launch_bounds__(kPlaceBlock) void expert_scan_kernel(uint32_t *__restrict__ table, uint32_t chunks,
                                                                  uint32_t experts, uint32_t *__restrict__ totals) {
    __shared__ uint4 sums[kScanSplits][kScanQuads];
    const uint32_t stride = table_stride(experts) / 4;
    const uint32_t q = threadIdx.x % kScanQuads, split = threadIdx.x / kScanQuads;
    const uint32_t quad = blockIdx.x * kScanQuads + q, lo = split * kScanRows;
    uint4 *const column = reinterpret_cast<uint4 *>(table) + (quad < stride ? quad : stride - 1);
    const auto add = [](uint4 &a, const uint4 &b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; };
    uint4 held[kScanRows], sum = make_uint4(0, 0, 0, 0), run = sum;
#pragma unroll
    for (uint32_t i = 0; i < kScanRows; ++i) {
        held[i] = column[static_cast<size_t>(lo + i < chunks ? lo + i : chunks - 1) * stride];
    }
#pragma unroll
    for (uint32_t i = 0; i < kScanRows; ++i) {
        if (lo + i >= chunks) held[i] = make_uint4(0, 0, 0, 0);
        add(sum, held[i]);
    }
    sums[split][q] = sum;
    __syncthreads();
    for (uint32_t i = 0; i < split; ++i) add(run, sums[i][q]);
    if (quad >= stride) return;
#pragma unroll
    for (uint32_t i = 0; i < kScanRows; ++i) {
        if (lo + i < chunks) column[static_cast<size_t>(lo + i) * stride] = run;
        add(run, held[i]);
    }
    if (split == kScanSplits - 1) reinterpret_cast<uint4 *>(totals)[quad] = run;
}

// Places of a chunk of slots: order[place] = slot, position[slot] = place
// (~place for a dropped slot).  A slot's place is
//   (slots of smaller keys) + (slots of its key in earlier chunks, waves and
//   rounds of its wave) + (lanes below it in its round with its key),
// so equal keys keep slot order whatever the waves' timing.  The last two terms
// are what an LDS add to the wave's counter of the key returns: like the pass
// kernel's local rank, this takes the lanes' same-address adds to be served
// in lane order, a measured property, here among up to 1025 counters and with
// lanes masked out, which the tests of this sort pin on the lane order test's
// patterns.  match: ranked by ballots instead (match_rank), whatever that order;
// 2^20 slots of 256 experts take 2.5 us more so, 8192 slots 4.3.  Dropped slots,
// often a long run of padding, are ranked by a ballot instead of 64 adds to one
// address.  A tile's slots are put in key order in LDS, so that order is written in runs
// (the sort of 2^20 slots of 256 experts takes 13.4 us so, 16.1 without).
// KEYS >= experts sizes the LDS.  Bound by the chain of round trips: ids and
// table, LDS counts, scans, writes: 8.9 us for 2^20 slots of 128 experts (12 MiB).
enum : int {
    kNoTable = 0,  // one workgroup that holds every slot in one tile
    kCounts = 1,   // every chunk's counts are in the table: each workgroup sums them
    kScanned = 2,  // the table's columns are scanned, their totals beside it
};

template <class ID, int ITEMS, int KEYS, int TABLE>
__global__ __launch_bounds__(kPlaceBlock) void expert_place_kernel(const ID *__restrict__ ids, size_t n, ID first,
                                                                   uint32_t experts, size_t chunk,
                                                                   const uint32_t *__restrict__ table,
                                                                   const uint32_t *__restrict__ totals, bool match,
                                                                   int32_t *__restrict__ order,
                                                                   int32_t *__restrict__ position,
                                                                   int32_t *__restrict__ offsets) {
    constexpr uint32_t kTile = kPlaceBlock * ITEMS;
    constexpr int kKeyBits = KEYS == 256 ? 9 : 11;  // of keys up to KEYS
    static_assert(kTile <= 0x10000 && KEYS <= kPlaceBlock && KEYS < 1 << kKeyBits);
    __shared__ uint32_t count[kPlaceWaves * (KEYS + 1)];  // [wave][key]
    __shared__ uint32_t base[KEYS + 1];                   // place of the next slot of a key
    __shared__ uint32_t delta[KEYS + 1];                  // a slot's place less its place in the tile
    __shared__ __attribute__((aligned(16))) uint32_t sorted[kTile];  // the tile in key order: slot in tile | key << 16
    __shared__ uint32_t wave_total[2][kPlaceWaves];
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const uint32_t keys = experts + 1;
    const size_t lo = blockIdx.x * chunk;
    const size_t hi = lo + chunk < n ? lo + chunk : n;

    uint32_t key[ITEMS], rank[ITEMS];
    const uint32_t mine = wave * 64 * ITEMS + lane;  // the thread's first slot in a tile
    const auto load_keys = [&](size_t tile) {
        ID id[ITEMS] = {};  // all in flight: beyond the chunk the last slot, not used
        if (tile < hi) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const size_t slot = tile + mine + i * 64;
                id[i] = ids[slot < hi ? slot : hi - 1];
            }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            key[i] = tile + mine + i * 64 < hi ? expert_key(id[i], first, experts) : 0xFFFFFFFFu;
        }
    };
    // The workgroup's sum of x below this thread, and all of it.
    const auto scan = [&](uint32_t x, uint32_t *wave_sum, uint32_t &all) {
        const uint32_t incl = wave_inclusive_sum(x);
        if (lane == 63) wave_sum[wave] = incl;
        __syncthreads();
        const uint32_t others = lane < kPlaceWaves ? wave_sum[lane] : 0u;
        all = group_sum_u32<64>(others);
        return group_sum_u32<64>(lane < wave ? others : 0u) + incl - x;
    };
    load_keys(lo);
    uint32_t total = 0, before = 0;  // of expert tid: all slots, slots of earlier chunks
    if constexpr (TABLE == kCounts) {
        // A thread sums four experts over every splits-th row; the threads'
        // sums meet in LDS.
        static_assert(kTile >= 4 * kPlaceBlock || TABLE != kCounts);
        const uint32_t stride = table_stride(experts);
        uint32_t quads = 16;
        while (quads * 4 < stride) quads *= 2;
        const uint32_t splits = kPlaceBlock / quads, quad = tid % quads, split = tid / quads;
        const uint4 *const column = reinterpret_cast<const uint4 *>(table) + (quad * 4 < stride ? quad : 0);
        uint4 all = make_uint4(0, 0, 0, 0), ahead = make_uint4(0, 0, 0, 0);
        constexpr uint32_t kRows = 8;  // in flight: beyond the table its last row, not added
        for (uint32_t b = split; b < gridDim.x; b += kRows * splits) {
            uint4 c[kRows];
#pragma unroll
            for (uint32_t i = 0; i < kRows; ++i) {
                const uint32_t row = b + i * splits < gridDim.x ? b + i * splits : gridDim.x - 1;
                c[i] = column[static_cast<size_t>(row) * (stride / 4)];
            }
#pragma unroll
            for (uint32_t i = 0; i < kRows; ++i) {
                const uint32_t m = b + i * splits < gridDim.x ? 0xFFFFFFFFu : 0u;
                const uint32_t m2 = b + i * splits < blockIdx.x ? 0xFFFFFFFFu : 0u;
                all.x += c[i].x & m, all.y += c[i].y & m, all.z += c[i].z & m, all.w += c[i].w & m;
                ahead.x += c[i].x & m2, ahead.y += c[i].y & m2, ahead.z += c[i].z & m2, ahead.w += c[i].w & m2;
            }
        }
        const auto meet = [&](const uint4 &part) {
            uint4 *const parts = reinterpret_cast<uint4 *>(sorted);
            parts[tid] = part;
            __syncthreads();
            uint32_t sum = 0;
            if (tid < experts) {
#pragma unroll 8
                for (uint32_t i = 0; i < splits; ++i) sum += sorted[i * quads * 4 + tid];
            }
            __syncthreads();
            return sum;
        };
        total = meet(all);
        before = meet(ahead);
    }
    if (TABLE == kScanned && tid < experts) {
        total = totals[tid];
        before = table[blockIdx.x * static_cast<size_t>(table_stride(experts)) + tid];
    }

    for (size_t tile = lo; tile == lo || tile < hi; tile += kTile) {
        for (uint32_t i = tid; i < kPlaceWaves * keys; i += kPlaceBlock) count[i] = 0;
        __syncthreads();
        uint32_t *const own = count + wave * keys;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (match) {
                rank[i] = match_rank<kKeyBits>(key[i], key[i] <= experts, own, 1u);
                continue;
            }
            if (key[i] < experts) rank[i] = atomicAdd(&own[key[i]], 1u);
            const uint64_t dropped = __ballot(key[i] == experts);
            if (dropped != 0) {
                uint32_t start = 0;
                if (lane == 0) start = atomicAdd(&own[experts], static_cast<uint32_t>(__popcll(dropped)));
                start = lane_value(start, 0);
                if (key[i] == experts) {
                    rank[i] = __builtin_amdgcn_mbcnt_hi(
                        static_cast<uint32_t>(dropped >> 32),
                        __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(dropped), start));
                }
            }
        }
        __syncthreads();

        // Where each key starts in the tile: an exclusive scan of its counts.
        uint32_t in_tile = 0, used_in_tile;
        if (tid < experts) {
#pragma unroll
            for (uint32_t w = 0; w < kPlaceWaves; ++w) in_tile += count[w * keys + tid];
        }
        const uint32_t local = scan(in_tile, wave_total[0], used_in_tile);
        if (tile == lo) {
            // And in the whole: the same scan of the totals.  The dropped
            // slots of earlier chunks are what is left of those chunks.
            uint32_t used = used_in_tile, start = local, ahead = 0;
            if constexpr (TABLE != kNoTable) {
                start = scan(total, wave_total[1], used);
                __syncthreads();
                scan(before, wave_total[1], ahead);
            }
            if (tid < experts) base[tid] = start + before;
            if (tid == 0) base[experts] = used + static_cast<uint32_t>(lo) - ahead;
            if (blockIdx.x == 0) {
                if (tid < experts) offsets[tid] = static_cast<int32_t>(start);
                if (tid == 0) offsets[experts] = static_cast<int32_t>(used);
            }
            __syncthreads();
        }
        // The waves' starts of each key in the tile.
        for (uint32_t e = tid; e < keys; e += kPlaceBlock) {
            uint32_t run = e < experts ? local : used_in_tile, c[kPlaceWaves];
#pragma unroll
            for (uint32_t w = 0; w < kPlaceWaves; ++w) c[w] = count[w * keys + e];
            const uint32_t at = base[e] - run;
            delta[e] = at;
#pragma unroll
            for (uint32_t w = 0; w < kPlaceWaves; ++w) {
                count[w * keys + e] = run;
                run += c[w];
            }
            base[e] = at + run;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t slot = mine + i * 64;
            if (key[i] <= experts) {
                const uint32_t local_place = own[key[i]] + rank[i], place = local_place + delta[key[i]];
                sorted[local_place] = slot | key[i] << 16;
                position[tile + slot] = static_cast<int32_t>(key[i] == experts ? ~place : place);
            }
        }
        const uint32_t here = hi - tile < kTile ? static_cast<uint32_t>(hi - tile) : kTile;
        if (tile + kTile < hi) load_keys(tile + kTile);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t p = tid + i * kPlaceBlock;
            if (p < here) {
                const uint32_t v = sorted[p];
                order[p + delta[v >> 16]] = static_cast<int32_t>(tile + (v & 0xFFFFu));
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Rows to their places and back
// ---------------------------------------------------------------------------
constexpr int kRowBlock = 256;

// A slot's row and whether the slot is in use; a place outside the rows is
// left alone (row = -1).
struct Slot {
    int64_t row;
    bool used;
};

__device__ __forceinline__ Slot slot_of(int32_t position, size_t num_rows) {
    const bool used = position >= 0;
    const uint32_t place = static_cast<uint32_t>(used ? position : ~position);
    return {place < num_rows ? static_cast<int64_t>(place) : int64_t{-1}, used};
}

// What a row kernel works on.  Spread: rows_out[place of slot (t, j)] =
// w[t, j] * x[t], zeros for a dropped slot.  Join: out[t] = sum over the used
// slots j of w[t, j] * rows_in[place of (t, j)], in float, in the order of j.
// Dots: dots[t, j] = <x[t], rows_in[place of (t, j)]> in float, 0 for a
// dropped slot.
template <class T>
struct RowWork {
    const T *x;
    size_t x_stride;
    const T *rows_in;
    size_t rows_in_stride;
    T *rows_out;
    size_t rows_out_stride;
    T *out;
    size_t out_stride;
    float *dots;
    const int32_t *position;
    const float *weights;
    size_t tokens;
    size_t num_rows;
    int width;
    int k;
    int lanes;   // narrow rows: threads of a row
    int chunks;  // wide rows: rounds of the lanes that cover a row
    int side;    // wide rows without dots: log2 of the waves side by side
    bool once;   // wide rows: rows_in is read past the caches' keeping
    unsigned clearing;    // spread: leading workgroups (lines of them in a grid of two dimensions) that only
                          // clear the rows that no slot names
    uint32_t clear_rows;  // rows that each of them takes at a time, at most kClearRows
};

// Zeros in the rows_out that no slot names, used or dropped, by workgroup
// `group` of `groups`: it marks the named ones of clear_rows rows in LDS, from
// all places, and clears the others.  The rest of the launch writes named rows
// only, so neither has to wait for the other.  Bound by the vector work on each
// place, some 90 cycles for 64 of them: 11 us for 65536 slots, while the rows take
// the memory's time (8192 x 8 x 2048 bfloat16 with dots: 91 us with and without).
constexpr uint32_t kClearRows = 65536;

template <class T>
__device__ __forceinline__ void clear_unnamed_rows(const RowWork<T> &a, size_t group, size_t groups) {
    constexpr int W = kVec<T>;
    constexpr int kDeep = 8;  // accesses of a thread in flight
    typedef int32_t Quad __attribute__((ext_vector_type(4), aligned(4)));
    __shared__ uint32_t named[kClearRows / 32];
    const uint32_t tid = threadIdx.x, lane = tid % 64;
    const size_t slots = a.tokens * static_cast<size_t>(a.k), quads = slots / 4;
    for (size_t lo = group * a.clear_rows; lo < a.num_rows; lo += groups * a.clear_rows) {
        const uint32_t rows = a.num_rows - lo < a.clear_rows ? static_cast<uint32_t>(a.num_rows - lo) : a.clear_rows;
        const uint32_t words = (rows + 31) / 32;
        for (uint32_t i = tid; i < words; i += kRowBlock) named[i] = 0;
        __syncthreads();
        const auto mark = [&](int32_t position) {
            const uint32_t r = static_cast<uint32_t>(position >= 0 ? position : ~position) - static_cast<uint32_t>(lo);
            if (r < rows) atomicOr(&named[r / 32], 1u << r % 32);
        };
        for (size_t q0 = tid; q0 < quads; q0 += kRowBlock * kDeep) {
            Quad v[kDeep];  // behind the end the last one again: a mark twice is a mark
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const size_t q = q0 + static_cast<size_t>(i) * kRowBlock;
                v[i] = reinterpret_cast<const Quad *>(a.position)[q < quads ? q : quads - 1];
            }
#pragma unroll
            for (int i = 0; i < kDeep; ++i) mark(v[i].x), mark(v[i].y), mark(v[i].z), mark(v[i].w);
        }
        if (tid < slots % 4) mark(a.position[quads * 4 + tid]);
        __syncthreads();
        for (uint32_t w0 = tid - lane; w0 < words; w0 += kRowBlock) {
            const uint32_t w = w0 + lane, have = rows - w * 32;  // rows of the lane's word, if it has any
            uint32_t left = 0;
            if (w < words) left = ~named[w] & (have < 32 ? (1u << have) - 1 : 0xFFFFFFFFu);
            for (uint64_t some = __ballot(left != 0); some != 0; some &= some - 1) {
                const int of = __builtin_ctzll(some);
                for (uint32_t m = lane_value(left, of); m != 0; m &= m - 1) {
                    const size_t row = lo + (w0 + static_cast<uint32_t>(of)) * 32 + static_cast<uint32_t>(__builtin_ctz(m));
                    const float zeros[W] = {};
                    for (int col = static_cast<int>(lane) * W; col < a.width; col += 64 * W) {
                        store_some<T, W>(a.rows_out + row * a.rows_out_stride + col, a.width - col, zeros);
                    }
                }
            }
        }
        __syncthreads();
    }
}

constexpr int kMaxBatch = 8;       // slots of a token whose rows are in flight together
constexpr int kMaxJoinBatch = 16;  // in a join with dots, which holds all of them

// Zeros in whole rows, `lanes` threads (a power of two) to a row: for the
// spreads whose time would not hide the search above.
template <class T>
__global__ __launch_bounds__(kRowBlock) void clear_rows_kernel(T *rows, size_t num_rows, int width, size_t stride,
                                                               int lanes) {
    constexpr int W = kVec<T>;
    const int per_block = kRowBlock / lanes;
    const float zeros[W] = {};
    for (size_t r = static_cast<size_t>(blockIdx.x) * per_block + threadIdx.x / lanes; r < num_rows;
         r += static_cast<size_t>(gridDim.x) * per_block) {
        for (int col = static_cast<int>(threadIdx.x) % lanes * W; col < width; col += lanes * W) {
            store_some<T, W>(rows + r * stride + col, width - col, zeros);
        }
    }
}

// Rows of more than kNarrow 16-byte accesses.  LANES threads hold 16-byte
// columns of a token's row: they read x once and write it k times, or read k
// rows (BATCH of them in flight) and write their sum once.  A token is the
// same for a whole wave: its places and weights are scalars.
// Without dots a wave takes one chunk of 64 columns of a token.  With dots the
// LANES threads take the whole row, chunk after chunk, since their products
// meet at the end, AT_ONCE chunks in flight together; a join with dots holds one
// batch (k <= BATCH).
// The loads of a batch are issued without a branch between them, which would
// wait for the one before: an unused slot reads a used one's row.
// The last access of a row is moved back to end with it where the width is no
// multiple of the access: its first elements are computed twice, to the same
// result, and counted once in the products.
// Bound by memory, which a plain copy moves at 4.9 - 5.7 TB/s: bfloat16 spread
// 16384 x 8 x 4096 217 us (5.6 TB/s), join 206 us (5.9, its output partly taken by
// the last-level cache; 224 us, 5.4, where that holds none of it), spread with dots
// 8192 x 8 x 2048 117 us (4.9), join with dots 60 us (5.6).  Row by row instead of
// in batches the join took 262 us, dots in a pass of their own 144 in all.
// a.once (ONCE without dots, where the branch would cost a small join 0.3 us of
// 3.5) reads rows_in with non-temporal loads, where the rows do not fit the
// last-level cache anyway: what the writes before and after leave there lasts
// longer.  Joins gain 12% so (234 -> 206 us), and a spread with dots gains it in
// the kernel that reads its result next (110 -> 98 us for both, 4093 x 2 x 4099
// float32); rows that fit are better kept (45 -> 47 us for 2048 x 8 x 2048).
// Non-temporal stores help the call alone and cost the next one as much.
constexpr int kNarrow = 32;

template <class T, int LANES, int BATCH, int AT_ONCE, bool SPREAD, bool WEIGHTED, bool DOTS, bool ONCE>
__global__ __launch_bounds__(kRowBlock) void wide_rows_kernel(const RowWork<T> a) {
    constexpr int W = kVec<T>;
    using Vec = typename VecOf<T, W>::type;
    constexpr int kPer = kRowBlock / LANES;
    constexpr int kWaves = LANES / 64;
    static_assert((LANES == 64 && AT_ONCE == 1) || (DOTS && LANES == kRowBlock));
    __shared__ float partial[kWaves > 1 ? BATCH : 1][kWaves > 1 ? kWaves : 1];
    const int lane = threadIdx.x % LANES;
    const int group = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / LANES);
    // Workgroup (x, y): without dots chunks x * 2^side ... and tokens y * (kPer /
    // 2^side) ..., 2^side waves side by side in a row; with dots tokens alone.
    if constexpr (SPREAD) {
        if ((DOTS ? blockIdx.x : blockIdx.y) < a.clearing) {
            const size_t across = DOTS ? 1 : gridDim.x;
            clear_unnamed_rows<T>(a, DOTS ? blockIdx.x : blockIdx.y * across + blockIdx.x, a.clearing * across);
            return;
        }
    }
    const unsigned ahead = SPREAD ? a.clearing : 0;
    const int side = DOTS ? 0 : a.side;
    const int first = DOTS ? 0 : static_cast<int>(blockIdx.x << side) + (group & ((1 << side) - 1));
    if (first >= a.chunks) return;
    const size_t block = (DOTS ? blockIdx.x : blockIdx.y) - ahead, blocks = (DOTS ? gridDim.x : gridDim.y) - ahead;
    for (size_t t = block * (kPer >> side) + (group >> side); t < a.tokens; t += blocks * (kPer >> side)) {
        float acc[W] = {};
        for (int j0 = 0; j0 < a.k; j0 += BATCH) {
            // Lane i of each wave loads slot j0 + i; the wave reads them as scalars.
            const int mine = j0 + static_cast<int>(threadIdx.x % 64);
            const size_t at = t * static_cast<size_t>(a.k) + (mine < a.k ? mine : a.k - 1);
            int32_t my_place = a.position[at];
            float my_weight = WEIGHTED ? a.weights[at] : 1.0f;
            asm volatile("" : "+v"(my_place), "+v"(my_weight));  // one wait for both loads
            Slot slot[BATCH];
            float w[BATCH];
            int64_t some = -1;  // the row of a used slot
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                slot[i] = slot_of(__builtin_amdgcn_readlane(my_place, i), a.num_rows);
                w[i] = __uint_as_float(lane_value(__float_as_uint(my_weight), i));
                if (j0 + i >= a.k) slot[i].row = -1;
                slot[i].used = slot[i].used & (slot[i].row >= 0);
                some = slot[i].used ? slot[i].row : some;
            }
            float dot[BATCH] = {};
            for (int c = first; c < (DOTS ? a.chunks : first + 1); c += AT_ONCE) {
                int begin[AT_ONCE], col[AT_ONCE];
                Vec raw[AT_ONCE][BATCH];
                float x[AT_ONCE][W];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    // Lanes behind the end read the last access, for nothing.
                    begin[u] = ((c + u) * LANES + lane) * W;
                    col[u] = begin[u] + W <= a.width ? begin[u] : a.width - W;
                    if constexpr (SPREAD || DOTS) load_vec<T, W>(a.x + t * a.x_stride + col[u], x[u]);
                }
                if constexpr (!SPREAD || DOTS) {
                    const auto load_rows = [&](auto load) {
#pragma unroll
                        for (int u = 0; u < AT_ONCE; ++u) {
#pragma unroll
                            for (int i = 0; i < BATCH; ++i) {
                                const auto row = static_cast<size_t>(slot[i].used ? slot[i].row : some);
                                raw[u][i] = load(reinterpret_cast<const Vec *>(a.rows_in + row * a.rows_in_stride + col[u]));
                            }
                        }
                    };
                    const auto past = [](const Vec *p) { return __builtin_nontemporal_load(p); };
                    const auto kept = [](const Vec *p) { return *p; };
                    if constexpr (DOTS) {
                        if (some >= 0 && a.once) load_rows(past);
                        if (some >= 0 && !a.once) load_rows(kept);
                    } else if (some >= 0) {
                        if constexpr (ONCE) load_rows(past);
                        if constexpr (!ONCE) load_rows(kept);
                    }
                }
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    const bool live = begin[u] < a.width;
                    if (SPREAD && live) {
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) {
                            if (slot[i].row < 0) continue;
                            float v[W];
#pragma unroll
                            for (int e = 0; e < W; ++e) {
                                v[e] = !slot[i].used ? 0.0f : WEIGHTED ? w[i] * x[u][e] : x[u][e];
                            }
                            store_vec<T, W>(a.rows_out + static_cast<size_t>(slot[i].row) * a.rows_out_stride + col[u],
                                            v);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        if ((SPREAD && !DOTS) || !slot[i].used) continue;
                        float f[W];
#pragma unroll
                        for (int e = 0; e < W; ++e) f[e] = static_cast<float>(raw[u][i][e]);
                        if constexpr (!SPREAD) {
#pragma unroll
                            for (int e = 0; e < W; ++e) {
                                acc[e] = WEIGHTED ? __builtin_fmaf(w[i], f[e], acc[e]) : acc[e] + f[e];
                            }
                        }
                        if constexpr (DOTS) {
                            if (col[u] == begin[u]) {
#pragma unroll
                                for (int e = 0; e < W; ++e) dot[i] = __builtin_fmaf(x[u][e], f[e], dot[i]);
                            } else {
#pragma unroll
                                for (int e = 0; e < W; ++e) {
                                    if (col[u] + e >= begin[u]) dot[i] = __builtin_fmaf(x[u][e], f[e], dot[i]);
                                }
                            }
                        }
                    }
                    if constexpr (!SPREAD) {
                        if (DOTS || j0 + BATCH >= a.k) {
                            if (live) store_vec<T, W>(a.out + t * a.out_stride + col[u], acc);
#pragma unroll
                            for (int e = 0; e < W; ++e) acc[e] = 0.0f;
                        }
                    }
                }
            }
            if constexpr (DOTS) {
                float total = 0.0f;
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const float sum = group_sum<64>(dot[i]);
                    if constexpr (kWaves > 1) {
                        if (lane % 64 == i) partial[i][lane / 64] = sum;
                    } else {
                        total = lane == i ? sum : total;
                    }
                }
                if constexpr (kWaves > 1) {
                    __syncthreads();
                    if (lane < BATCH) {
#pragma unroll
                        for (int i = 0; i < kWaves; ++i) total += partial[lane][i];
                    }
                }
                // An unused slot's sum is 0: nothing was added to it.
                if (lane < BATCH && j0 + lane < a.k) a.dots[t * static_cast<size_t>(a.k) + j0 + lane] = total;
                if constexpr (kWaves > 1) __syncthreads();
            }
        }
    }
}

// Rows of at most kNarrow 16-byte accesses: a.lanes threads (a power of two)
// take a token's row, an access each, and add their products up in pairs.
// 65536 x 8 x 128 bfloat16: join 36 us, spread with dots 67 us (4.3 TB/s both).
template <class T, bool SPREAD, bool WEIGHTED, bool DOTS>
__global__ __launch_bounds__(kRowBlock) void narrow_rows_kernel(const RowWork<T> a) {
    constexpr int W = kVec<T>;
    if constexpr (SPREAD) {
        if (blockIdx.x < a.clearing) {
            clear_unnamed_rows<T>(a, blockIdx.x, a.clearing);
            return;
        }
    }
    const unsigned ahead = SPREAD ? a.clearing : 0;
    const int per_block = kRowBlock / a.lanes;
    const int lane = static_cast<int>(threadIdx.x) % a.lanes;
    const int col = lane * W, have = a.width - col;  // have <= 0: a lane beyond the row
    for (size_t t = static_cast<size_t>(blockIdx.x - ahead) * per_block + threadIdx.x / a.lanes; t < a.tokens;
         t += static_cast<size_t>(gridDim.x - ahead) * per_block) {
        float x[W], acc[W] = {};
        if constexpr (SPREAD || DOTS) load_some<T, W>(a.x + t * a.x_stride + col, have, x);
        for (int j = 0; j < a.k; ++j) {
            const size_t s = t * static_cast<size_t>(a.k) + j;
            const Slot slot = slot_of(a.position[s], a.num_rows);
            const bool used = slot.row >= 0 && slot.used;
            const float w = WEIGHTED ? a.weights[s] : 1.0f;
            if constexpr (SPREAD) {
                if (slot.row >= 0) {
                    float v[W];
#pragma unroll
                    for (int i = 0; i < W; ++i) v[i] = !slot.used ? 0.0f : WEIGHTED ? w * x[i] : x[i];
                    store_some<T, W>(a.rows_out + static_cast<size_t>(slot.row) * a.rows_out_stride + col, have, v);
                }
            }
            if constexpr (!SPREAD || DOTS) {
                float dot = 0.0f;
                if (used) {
                    float f[W];
                    load_some<T, W>(a.rows_in + static_cast<size_t>(slot.row) * a.rows_in_stride + col, have, f);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        if constexpr (!SPREAD) acc[i] = WEIGHTED ? __builtin_fmaf(w, f[i], acc[i]) : acc[i] + f[i];
                        if constexpr (DOTS) dot = __builtin_fmaf(x[i], f[i], dot);
                    }
                }
                if constexpr (DOTS) {
                    for (int step = a.lanes / 2; step > 0; step /= 2) dot += __shfl_xor(dot, step, 64);
                    if (lane == 0) a.dots[s] = dot;
                }
            }
        }
        if constexpr (!SPREAD) store_some<T, W>(a.out + t * a.out_stride + col, have, acc);
    }
}

// Dots alone, for wide joins of more than kMaxJoinBatch slots, whose kernel does
// not take them along (10 slots would take 157 us so for 8192 x 2048 bfloat16,
// 72 in one pass).  A wave takes a slot.
template <class T>
__global__ __launch_bounds__(kRowBlock) void dot_rows_kernel(const RowWork<T> a) {
    constexpr int W = kVec<T>;
    constexpr int kWaves = kRowBlock / 64;
    const int lane = threadIdx.x % 64;
    const size_t slots = a.tokens * static_cast<size_t>(a.k);
    for (size_t s = static_cast<size_t>(blockIdx.x) * kWaves + threadIdx.x / 64; s < slots;
         s += static_cast<size_t>(gridDim.x) * kWaves) {
        const Slot slot = slot_of(a.position[s], a.num_rows);
        float acc = 0.0f;
        if (slot.row >= 0 && slot.used) {
            const T *x = a.x + (s / a.k) * a.x_stride;
            const T *row = a.rows_in + static_cast<size_t>(slot.row) * a.rows_in_stride;
            for (int col = lane * W; col < a.width; col += 64 * W) {
                float f[W], h[W];
                load_some<T, W>(x + col, a.width - col, f);
                load_some<T, W>(row + col, a.width - col, h);
#pragma unroll
                for (int i = 0; i < W; ++i) acc = __builtin_fmaf(f[i], h[i], acc);
            }
        }
        acc = group_sum<64>(acc);
        if (lane == 0) a.dots[s] = acc;
    }
}

}  // namespace rs
