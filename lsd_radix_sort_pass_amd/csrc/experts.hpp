// experts.hpp -- gfx950 kernels of the mixture-of-experts calls: top-k
// routing of router logits, the stable sort of (token, choice) slots by
// expert, and the movement of token rows to their sorted places and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

namespace rs {

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------
using bf16 = __bf16;
using f16 = _Float16;

template <class T, int N>
struct VecOf {
    // Only element alignment is assumed: gfx950 serves unaligned 16-byte
    // global accesses, so odd widths and strides take the same wide path.
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte access

template <class T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = static_cast<float>(*p);
    } else {
        const auto v = *reinterpret_cast<const typename VecOf<T, N>::type *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = static_cast<float>(v[i]);
    }
}

// Rounds to nearest even where T is narrower than float: the one rounding
// of a result, after its sum in float.
template <class T, int N>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[N]) {
    if constexpr (N == 1) {
        *p = static_cast<T>(f[0]);
    } else {
        typename VecOf<T, N>::type v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = static_cast<T>(f[i]);
        *reinterpret_cast<typename VecOf<T, N>::type *>(p) = v;
    }
}

// The N elements at p, of which only the first `have` exist (zeros beyond).
template <class T, int N>
__device__ __forceinline__ void load_some(const T *p, int have, float (&f)[N]) {
    if (have >= N) {
        load_vec<T, N>(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = i < have ? static_cast<float>(p[i]) : 0.0f;
    }
}

template <class T, int N>
__device__ __forceinline__ void store_some(T *p, int have, const float (&f)[N]) {
    if (have >= N) {
        store_vec<T, N>(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < have) p[i] = static_cast<T>(f[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Reductions over a group of 16 or 64 consecutive lanes; every lane of the
// group gets the result.  All 64 lanes of the wave must be active.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, 0xF, 0xF, false));
}

template <int G, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t x, F f) {
    static_assert(G == 16 || G == 64);
    x = f(x, dpp<0xB1>(x));   // quad_perm: lane ^ 1
    x = f(x, dpp<0x4E>(x));   // quad_perm: lane ^ 2
    x = f(x, dpp<0x141>(x));  // row_half_mirror: the other quad of 8
    x = f(x, dpp<0x140>(x));  // row_mirror: the other half of 16
    if constexpr (G == 64) {
        const uint32_t a = f(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 0)),
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 16)));
        const uint32_t b = f(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 32)),
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 48)));
        x = f(a, b);
    }
    return x;
}

template <int G>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int G>
__device__ __forceinline__ uint32_t group_min_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

template <int G>
__device__ __forceinline__ uint32_t group_sum_u32(uint32_t x) {
    return group_reduce<G>(x, [](uint32_t a, uint32_t b) { return a + b; });
}

template <int G>
__device__ __forceinline__ float group_max(float x) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
constexpr int kRouteBlock = 256;

// Rank of a logit as an unsigned integer: a larger logit has a larger rank,
// -0 equals +0, every NaN ranks above every number, and -inf (an expert that
// the row may not use) has rank 0, below every finite value.  It keeps the
// value: ranked_value undoes it.
__device__ __forceinline__ uint32_t rank16(uint32_t bits, uint32_t inf) {
    if (bits == 0x8000u) bits = 0;
    if (bits == (inf | 0x8000u)) return 0;
    if ((bits & 0x7FFFu) > inf) return 0xFFFFu;
    return (bits & 0x8000u) ? (~bits & 0xFFFFu) : (bits | 0x8000u);
}

__device__ __forceinline__ uint32_t unrank16(uint32_t rank) {
    return (rank & 0x8000u) ? (rank ^ 0x8000u) : (~rank & 0xFFFFu);
}

__device__ __forceinline__ uint32_t rank_of(float x) {
    uint32_t bits = __float_as_uint(x);
    if (bits == 0x80000000u) bits = 0;
    if (bits == 0xFF800000u) return 0;
    if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
}
__device__ __forceinline__ uint32_t rank_of(f16 x) { return rank16(__builtin_bit_cast(uint16_t, x), 0x7C00u); }
__device__ __forceinline__ uint32_t rank_of(bf16 x) { return rank16(__builtin_bit_cast(uint16_t, x), 0x7F80u); }

template <class T>
__device__ __forceinline__ float ranked_value(uint32_t rank) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float((rank & 0x80000000u) ? (rank ^ 0x80000000u) : ~rank);
    } else {
        return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(unrank16(rank))));
    }
}

enum : int { kGateSoftmax = 0, kGateSigmoid = 1 };

// 1 / (1 + exp(-l)), and its complement as sigmoid(-l); exp only of numbers
// <= 0, so neither end overflows.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-__builtin_fabsf(l));
    return (l >= 0.0f || l != l ? 1.0f : e) / (1.0f + e);
}

// G lanes hold a row's logits, V each: lane g holds the elements
// (c * G + g) * W + w of chunk c.  k rounds take the group's largest rank;
// lane j keeps round j's winner, so k <= G.
// 16-bit logits carry 0xFFFF - index below the rank: one maximum finds the
// value and, among equals, the lowest index.  32-bit logits take a second
// reduction for the index.
template <class T, int G, int V>
__global__ __launch_bounds__(kRouteBlock) void route_topk_kernel(const T *__restrict__ logits, size_t tokens,
                                                                 int experts, size_t stride, int k, int gate,
                                                                 int renormalize, float scale,
                                                                 float *__restrict__ weights,
                                                                 int32_t *__restrict__ chosen) {
    constexpr int W = V < kVec<T> ? V : kVec<T>;
    constexpr int C = V / W;
    constexpr int kRows = kRouteBlock / G;
    constexpr bool kPacked = sizeof(T) == 2;
    const int g = threadIdx.x % G;
    for (size_t first = static_cast<size_t>(blockIdx.x) * kRows; first < tokens;
         first += static_cast<size_t>(gridDim.x) * kRows) {
        const size_t mine = first + threadIdx.x / G;
        const bool live = mine < tokens;
        const T *row = logits + (live ? mine : tokens - 1) * stride;

        uint32_t rank[V];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i0 = (c * G + g) * W;
            T raw[W];
            if (i0 + W <= experts) {
                __builtin_memcpy(raw, row + i0, sizeof(raw));
#pragma unroll
                for (int w = 0; w < W; ++w) rank[c * W + w] = rank_of(raw[w]);
            } else {
#pragma unroll
                for (int w = 0; w < W; ++w) rank[c * W + w] = i0 + w < experts ? rank_of(row[i0 + w]) : 0u;
            }
            if constexpr (kPacked) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t r = rank[c * W + w];
                    rank[c * W + w] = r ? (r << 16) | (0xFFFFu - static_cast<uint32_t>(i0 + w)) : 0u;
                }
            }
        }

        const auto value = [&](uint32_t r) { return ranked_value<T>(kPacked ? r >> 16 : r); };
        const auto best_of = [&]() {
            uint32_t b = rank[0];
#pragma unroll
            for (int v = 1; v < V; ++v) b = rank[v] > b ? rank[v] : b;
            return group_max_u32<G>(b);
        };

        uint32_t best = best_of();
        const float top = value(best);
        float total = 0.0f;  // softmax over the whole row: sum of exp(l - top)
        if (gate == kGateSoftmax && !renormalize) {
#pragma unroll
            for (int v = 0; v < V; ++v) total += rank[v] ? expf(value(rank[v]) - top) : 0.0f;
            total = group_sum<G>(total);
        }

        uint32_t my_rank = 0, my_index = 0;
        for (int j = 0; j < k; ++j) {
            if (j > 0) best = best_of();
            if constexpr (kPacked) {
#pragma unroll
                for (int v = 0; v < V; ++v) rank[v] = rank[v] == best ? 0u : rank[v];
                if (g == j) {
                    my_rank = best;
                    my_index = 0xFFFFu - (best & 0xFFFFu);
                }
            } else {
                uint32_t at = 0xFFFFFFFFu;
#pragma unroll
                for (int v = V - 1; v >= 0; --v) {
                    const uint32_t i = static_cast<uint32_t>(((v / W) * G + g) * W + v % W);
                    at = rank[v] == best ? i : at;
                }
                at = group_min_u32<G>(at);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t i = static_cast<uint32_t>(((v / W) * G + g) * W + v % W);
                    rank[v] = i == at ? 0u : rank[v];
                }
                if (g == j) {
                    my_rank = best;
                    my_index = at;
                }
            }
        }

        // Lane j < k: slot j.  Rank 0: no expert was left to choose.
        const bool taken = g < k && my_rank != 0;
        const float l = value(my_rank);
        float w = 0.0f;
        if (gate == kGateSoftmax) {
            w = taken ? expf(l - top) : 0.0f;
            if (renormalize) total = group_sum<G>(w);
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
            chosen[at] = taken ? static_cast<int32_t>(my_index) : -1;
        }
    }
}

// Gradient of the router logits.  With p the gate's values, u = p / (sum of
// the chosen p), h the incoming gradient and a_i the sum of h over the slots
// that chose i:
//   softmax                dl_i = scale * p_i * (a_i - sum_j h_j p_j)
//   softmax, renormalized  dl_i = scale * u_i * (a_i - sum_j h_j u_j), chosen i only
//   sigmoid                dl_i = scale * a_i * p_i * (1 - p_i), chosen i only
//   sigmoid, renormalized  dl_i = scale * u_i * (a_i - sum_j h_j u_j) * (1 - p_i)
// Only the first needs the whole row; the others read the k chosen logits.
// Lane j < k of the group holds slot j; the slots' terms reach the lanes that
// hold their elements through LDS.
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
    for (size_t first = static_cast<size_t>(blockIdx.x) * kRows; first < tokens;
         first += static_cast<size_t>(gridDim.x) * kRows) {
        const size_t mine = first + sub;
        const bool live = mine < tokens;
        const size_t r = live ? mine : tokens - 1;
        const T *row = logits + r * stride;

        float p[V];
        float top = 0.0f, total = 1.0f;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int i0 = (c * G + g) * W;
                float f[W];
                load_some<T, W>(row + i0, experts - i0, f);
#pragma unroll
                for (int w = 0; w < W; ++w) p[c * W + w] = i0 + w < experts ? f[w] : -__builtin_inff();
            }
            top = p[0];
#pragma unroll
            for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, p[v]);
            top = group_max<G>(top);
            total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = p[v] == -__builtin_inff() ? 0.0f : expf(p[v] - top);
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
                    f[w] = p[c * W + w] == 0.0f ? 0.0f : scale * (q * (a - mean));
                } else {
                    f[w] = scale * a;
                }
            }
            if (live && i0 < experts) store_some<T, W>(out + i0, experts - i0, f);
        }
        __syncthreads();
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

// Keys of each workgroup's chunk of slots, counted in LDS:
// table[key][workgroup].
template <class ID>
__global__ __launch_bounds__(kPlaceBlock) void expert_count_kernel(const ID *__restrict__ ids, size_t n, ID first,
                                                                   uint32_t experts, size_t chunk,
                                                                   uint32_t *__restrict__ table) {
    __shared__ uint32_t count[kMaxExperts + 1];
    for (uint32_t e = threadIdx.x; e <= experts; e += kPlaceBlock) count[e] = 0;
    __syncthreads();
    const size_t lo = blockIdx.x * chunk;
    const size_t hi = lo + chunk < n ? lo + chunk : n;
    for (size_t i = lo + threadIdx.x; i < hi; i += kPlaceBlock) atomicAdd(&count[expert_key(ids[i], first, experts)], 1u);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e <= experts; e += kPlaceBlock) table[e * gridDim.x + blockIdx.x] = count[e];
}

// Places of a chunk of slots: order[place] = slot, position[slot] = place
// (~place for a dropped slot).  A slot's place is
//   (slots of smaller keys) + (slots of its key in earlier chunks, waves and
//   rounds of its wave) + (lanes below it in its round with its key),
// so equal keys keep slot order whatever the waves' timing.  The lanes of a
// round that share a key find each other by one ballot per key bit.
// Without a table the grid is one workgroup that holds every slot.
template <class ID, int ITEMS, bool TABLE>
__global__ __launch_bounds__(kPlaceBlock) void expert_place_kernel(const ID *__restrict__ ids, size_t n, ID first,
                                                                   uint32_t experts, int key_bits, size_t chunk,
                                                                   const uint32_t *__restrict__ table,
                                                                   int32_t *__restrict__ order,
                                                                   int32_t *__restrict__ position,
                                                                   int32_t *__restrict__ offsets) {
    __shared__ uint32_t count[kPlaceWaves * (kMaxExperts + 1)];
    __shared__ uint32_t base[kMaxExperts + 1];    // first place of the chunk's slots of a key
    __shared__ uint32_t wave_total[kPlaceWaves];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t keys = experts + 1;
    constexpr size_t kTile = static_cast<size_t>(kPlaceBlock) * ITEMS;
    const size_t lo = blockIdx.x * chunk;
    const size_t hi = lo + chunk < n ? lo + chunk : n;

    uint32_t total = 0, before = 0;  // of key threadIdx.x: all slots, slots of earlier chunks
    if constexpr (TABLE) {
        // A wave sums a key's row of the table.
        for (uint32_t e = wave; e < keys; e += kPlaceWaves) {
            uint32_t all = 0, ahead = 0;
            for (uint32_t b = lane; b < gridDim.x; b += 64) {
                const uint32_t c = table[e * gridDim.x + b];
                all += c;
                ahead += b < blockIdx.x ? c : 0u;
            }
            all = group_sum_u32<64>(all);
            ahead = group_sum_u32<64>(ahead);
            if (lane == 0) {
                count[e] = all;
                base[e] = ahead;
            }
        }
        __syncthreads();
        if (threadIdx.x < experts) {
            total = count[threadIdx.x];
            before = base[threadIdx.x];
        }
        __syncthreads();
    }

    for (size_t tile = lo; tile < hi || (!TABLE && tile == lo); tile += kTile) {
        for (uint32_t i = threadIdx.x; i < kPlaceWaves * keys; i += kPlaceBlock) count[i] = 0;
        __syncthreads();
        uint32_t key[ITEMS], rank[ITEMS];
        const size_t mine = tile + static_cast<size_t>(wave) * 64 * ITEMS + lane;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const size_t slot = mine + i * 64;
            key[i] = slot < hi ? expert_key(ids[slot], first, experts) : 0xFFFFFFFFu;
        }
        uint32_t *const own = count + wave * keys;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const bool live = key[i] != 0xFFFFFFFFu;
            uint64_t same = __ballot(live);
            for (int bit = 0; bit < key_bits; ++bit) {
                const bool one = (key[i] >> bit) & 1u;
                const uint64_t ones = __ballot(one);
                same &= one ? ones : ~ones;
            }
            const uint32_t below = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(same >> 32),
                                                             __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(same), 0u));
            uint32_t start = 0;
            if (live && below == 0) start = atomicAdd(&own[key[i]], static_cast<uint32_t>(__popcll(same)));
            const int leader = live ? __ffsll(static_cast<unsigned long long>(same)) - 1 : 0;
            rank[i] = __shfl(start, leader) + below;
        }
        __syncthreads();

        if (tile == lo) {
            // Bases: an exclusive scan of the keys' totals.
            if constexpr (!TABLE) {
                if (threadIdx.x < experts) {
                    for (int w = 0; w < kPlaceWaves; ++w) total += count[w * keys + threadIdx.x];
                }
            }
            uint32_t incl = threadIdx.x < experts ? total : 0u;
            const uint32_t own_total = incl;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t up = __shfl_up(incl, d);
                if (lane >= d) incl += up;
            }
            if (lane == 63) wave_total[wave] = incl;
            __syncthreads();
            uint32_t prior = 0, sum = 0;
            for (int w = 0; w < kPlaceWaves; ++w) {
                prior += w < wave ? wave_total[w] : 0u;
                sum += wave_total[w];
            }
            const uint32_t start = prior + incl - own_total;
            if (threadIdx.x < experts) base[threadIdx.x] = start + before;
            if (threadIdx.x == 0) base[experts] = sum + (TABLE ? base[experts] : 0u);
            if (blockIdx.x == 0) {
                if (threadIdx.x < experts) offsets[threadIdx.x] = static_cast<int32_t>(start);
                if (threadIdx.x == 0) offsets[experts] = static_cast<int32_t>(sum);
            }
            __syncthreads();
        }
        // Each wave's first place per key; the next tile starts behind the last.
        for (uint32_t e = threadIdx.x; e < keys; e += kPlaceBlock) {
            uint32_t run = base[e];
            for (int w = 0; w < kPlaceWaves; ++w) {
                const uint32_t c = count[w * keys + e];
                count[w * keys + e] = run;
                run += c;
            }
            base[e] = run;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const size_t slot = mine + i * 64;
            if (slot < hi) {
                const uint32_t place = own[key[i]] + rank[i];
                order[place] = static_cast<int32_t>(slot);
                position[slot] = static_cast<int32_t>(key[i] == experts ? ~place : place);
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

// rows[place of slot (t, j)] = w[t, j] * x[t]; zeros for a dropped slot.
// A group of `lanes` threads takes a 16-byte column of a token and writes it
// k times: x is read once.
template <class T, bool WEIGHTED>
__global__ __launch_bounds__(kRowBlock) void spread_rows_kernel(const T *__restrict__ x, size_t tokens, int width,
                                                                size_t x_stride, const int32_t *__restrict__ position,
                                                                const float *__restrict__ weights, int k,
                                                                T *__restrict__ rows, size_t num_rows,
                                                                size_t rows_stride, int lanes, int chunks) {
    constexpr int W = kVec<T>;
    const int per_block = kRowBlock / lanes;
    const size_t units = tokens * static_cast<size_t>(chunks);
    for (size_t u = static_cast<size_t>(blockIdx.x) * per_block + threadIdx.x / lanes; u < units;
         u += static_cast<size_t>(gridDim.x) * per_block) {
        const size_t t = u / chunks;
        const int col = (static_cast<int>(u % chunks) * lanes + static_cast<int>(threadIdx.x % lanes)) * W;
        const int have = width - col;
        if (have <= 0) continue;
        float f[W];
        load_some<T, W>(x + t * x_stride + col, have, f);
        for (int j = 0; j < k; ++j) {
            const size_t s = t * static_cast<size_t>(k) + j;
            const Slot slot = slot_of(position[s], num_rows);
            if (slot.row < 0) continue;
            float v[W];
            const float w = WEIGHTED ? weights[s] : 1.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = slot.used ? (WEIGHTED ? w * f[i] : f[i]) : 0.0f;
            store_some<T, W>(rows + static_cast<size_t>(slot.row) * rows_stride + col, have, v);
        }
    }
}

// out[t] = sum over the used slots j of w[t, j] * rows[place of (t, j)], in
// float, in the order of j.
template <class T, bool WEIGHTED>
__global__ __launch_bounds__(kRowBlock) void join_rows_kernel(const T *__restrict__ rows, size_t num_rows,
                                                              size_t rows_stride, const int32_t *__restrict__ position,
                                                              const float *__restrict__ weights, int k,
                                                              T *__restrict__ out, size_t tokens, int width,
                                                              size_t out_stride, int lanes, int chunks) {
    constexpr int W = kVec<T>;
    const int per_block = kRowBlock / lanes;
    const size_t units = tokens * static_cast<size_t>(chunks);
    for (size_t u = static_cast<size_t>(blockIdx.x) * per_block + threadIdx.x / lanes; u < units;
         u += static_cast<size_t>(gridDim.x) * per_block) {
        const size_t t = u / chunks;
        const int col = (static_cast<int>(u % chunks) * lanes + static_cast<int>(threadIdx.x % lanes)) * W;
        const int have = width - col;
        if (have <= 0) continue;
        float acc[W] = {};
        for (int j = 0; j < k; ++j) {
            const size_t s = t * static_cast<size_t>(k) + j;
            const Slot slot = slot_of(position[s], num_rows);
            if (slot.row < 0 || !slot.used) continue;
            float f[W];
            load_some<T, W>(rows + static_cast<size_t>(slot.row) * rows_stride + col, have, f);
            const float w = WEIGHTED ? weights[s] : 1.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = WEIGHTED ? __builtin_fmaf(w, f[i], acc[i]) : acc[i] + f[i];
        }
        store_some<T, W>(out + t * out_stride + col, have, acc);
    }
}

// dots[t, j] = <x[t], rows[place of (t, j)]> in float, 0 for a dropped slot.
// A wave takes a slot.
template <class T>
__global__ __launch_bounds__(kRowBlock) void dot_rows_kernel(const T *__restrict__ x, size_t tokens, int width,
                                                             size_t x_stride, const T *__restrict__ rows,
                                                             size_t num_rows, size_t rows_stride,
                                                             const int32_t *__restrict__ position, int k,
                                                             float *__restrict__ dots) {
    constexpr int W = kVec<T>;
    const int lane = threadIdx.x % 64;
    const size_t slots = tokens * static_cast<size_t>(k);
    constexpr int kWaves = kRowBlock / 64;
    for (size_t s = static_cast<size_t>(blockIdx.x) * kWaves + threadIdx.x / 64; s < slots;
         s += static_cast<size_t>(gridDim.x) * kWaves) {
        const Slot slot = slot_of(position[s], num_rows);
        float acc = 0.0f;
        if (slot.row >= 0 && slot.used) {
            const T *a = x + (s / k) * x_stride;
            const T *b = rows + static_cast<size_t>(slot.row) * rows_stride;
            for (int col = lane * W; col < width; col += 64 * W) {
                float f[W], h[W];
                load_some<T, W>(a + col, width - col, f);
                load_some<T, W>(b + col, width - col, h);
#pragma unroll
                for (int i = 0; i < W; ++i) acc = __builtin_fmaf(f[i], h[i], acc);
            }
        }
        acc = group_sum<64>(acc);
        if (lane == 0) dots[s] = acc;
    }
}

}  // namespace rs
