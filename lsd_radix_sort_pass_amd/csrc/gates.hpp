// gates.hpp -- gfx950 kernels between the experts' products: gated rows
//   h = act(a) b,  a row of 2 width elements holding a, then b,
// their gradients
//   da = g b act'(a),  db = g act(a),
// and rows in 8 bits with a scale for each 128 elements.  All of them pass once
// over their rows and are bound by memory.
#pragma once

#include "products.hpp"

namespace rs {

enum Act : int { kActSilu = 0, kActGelu = 1 };

// act(a) and act'(a).  silu: a s, s (1 + a (1 - s)) with s = sigmoid(a).  gelu:
// a F(a), F(a) + a f(a), with the normal distribution F (by its complement, which
// keeps its digits for negative a) and density f.
struct Activated {
    float value, slope;
};

// PRECISE: the exponential to its last digits, for rows of 32 bits; for those of 16, the
// machine's own, whose error grows with its argument: silu's 2^-21 at |a| = 8, 2^-18 at 87,
// gelu's, with the argument's own, 2^-20 at 4, 2^-17 at 13.  Results in 16 and 8 bits
// hide it; the scales of the latter carry it where a block's largest comes of so
// negative an a.  (With the digits that it lacks, 32768 x 2 * 2048 bfloat16 to 8 bits take 75 us where it
// takes 60, for scales of values whose own half step is 2^-4.)
template <int ACT, bool PRECISE>
__device__ __forceinline__ Activated activate(float a) {
    if constexpr (ACT == kActSilu) {
        const float size = __builtin_fabsf(a);
        const float e = PRECISE ? expf(-size) : __expf(-size);  // at most 1
        const float up = PRECISE ? 1.0f / (1.0f + e) : __builtin_amdgcn_rcpf(1.0f + e), down = e * up;
        const float s = a < 0.0f ? down : up, rest = a < 0.0f ? up : down;
        return {a * s, s + a * s * rest};
    } else if constexpr (PRECISE) {
        const float cdf = 0.5f * erfcf(-0.70710678f * a);
        const float density = 0.39894228f * expf(-0.5f * a * a);
        return {a * cdf, cdf + a * density};
    } else {
        // F(-|a|) = exp(-a^2 / 2) P(t), t = 1 / (1 + 0.4 |a| / sqrt 2): P the polynomial of the eighth
        // degree whose largest relative error for |a| up to 13.6 is least; with these constants it is
        // 2.0e-7, and 4.7e-7 worked out in float32.  (By
        // erfc, whose branches a wave takes both, the vector units bound the kernel:
        // 32768 x 2 * 2048 bfloat16 102 us, 70 so.)
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28284271f, __builtin_fabsf(a), 1.0f));
        const float e = __builtin_amdgcn_exp2f(-0.72134752f * (a * a));
        float y = 0.0365139591f;
        y = __builtin_fmaf(y, t, -0.195931294f);
        y = __builtin_fmaf(y, t, 0.343683708f);
        y = __builtin_fmaf(y, t, -0.194559737f);
        y = __builtin_fmaf(y, t, 0.214550314f);
        y = __builtin_fmaf(y, t, 0.0629367452f);
        y = __builtin_fmaf(y, t, 0.120794151f);
        y = __builtin_fmaf(y, t, 0.111971799f);
        y = __builtin_fmaf(y, t, 4.0284266e-05f);
        const float tail = y * e, cdf = a < 0.0f ? tail : 1.0f - tail;
        return {a * cdf, cdf + a * (0.39894228f * e)};
    }
}

// n / d for n < 2^31: n * ceil(2^(31 + L) / d) >> (31 + L), 2^L the least power of
// two that is at least d.
struct Divider {
    uint32_t multiplier, shift;
};

__device__ __forceinline__ uint32_t divide(uint32_t n, Divider d) {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.multiplier) >> d.shift);
}

struct GateWork {
    const void *rows, *grad;  // (num_rows, 2 width); (num_rows, width)
    void *out;                // (num_rows, width); of the gradient (num_rows, 2 width)
    size_t rows_stride, grad_stride, out_stride;
    float *scales;  // 8 bits: [blocks][num_rows]
    const int32_t *offsets;
    int experts;
    size_t num_rows;
    int width;
    bool clear;
    int chunks;  // of a row, 16 bytes of an input each (8 bits: scale blocks)
};

// The rows that belong to an expert.
__device__ __forceinline__ RowSpan live_rows(const int32_t *offsets, int experts, int num_rows) {
    if (offsets == nullptr) return {0, num_rows};
    const int lo = row_bound(offsets, 0, num_rows), hi = row_bound(offsets, experts, num_rows);
    return {lo, hi < lo ? lo : hi};
}

constexpr int kGateBlock = 256;

// V elements of each half a thread (16 bytes; one where a row has fewer).  The last
// ones of a row begin V before its end: elements of two threads get the same value
// from both, and no load or store sits in a branch.
template <class T, int V, int ACT, bool BACKWARD>
__global__ __launch_bounds__(kGateBlock) void gate_kernel(const GateWork w, const Divider by_chunks) {
    const RowSpan live = live_rows(w.offsets, w.experts, static_cast<int>(w.num_rows));
    const size_t units = w.num_rows * static_cast<size_t>(w.chunks);
    const size_t step = static_cast<size_t>(gridDim.x) * kGateBlock;
    for (size_t u = static_cast<size_t>(blockIdx.x) * kGateBlock + threadIdx.x; u < units; u += step) {
        const size_t r = units <= 0x7FFFFFFFu ? divide(static_cast<uint32_t>(u), by_chunks) : u / w.chunks;
        int c = static_cast<int>(u - r * w.chunks) * V;
        c = c < w.width - V ? c : w.width - V;
        const int row = static_cast<int>(r);
        const bool has = row >= live.lo && row < live.hi;
        float a[V], b[V], g[V], x[V], y[V];
        T *out = static_cast<T *>(w.out) + r * w.out_stride + c;
        if (!has) {
            if (!w.clear) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = y[i] = 0.0f;
        } else {
            const T *in = static_cast<const T *>(w.rows) + r * w.rows_stride + c;
            load_vec<T, V>(in, a);
            load_vec<T, V>(in + w.width, b);
            if constexpr (BACKWARD) load_vec<T, V>(static_cast<const T *>(w.grad) + r * w.grad_stride + c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Activated t = activate<ACT, std::is_same_v<T, float>>(a[i]);
                if constexpr (BACKWARD) {
                    x[i] = g[i] * b[i] * t.slope;
                    y[i] = g[i] * t.value;
                } else {
                    x[i] = t.value * b[i];
                }
            }
        }
        store_vec<T, V>(out, x);
        if constexpr (BACKWARD) store_vec<T, V>(out + w.width, y);
    }
}

// ---------------------------------------------------------------------------
// Rows to 8 bits.  A block of 128 elements has scale m / 448, m its largest
// finite size, at least 2^-100 (so that no scale is 0 and each has an inverse),
// and each element becomes e4m3(x / scale), the quotient rounded once to float32
// before; what is not finite becomes NaN.
// ---------------------------------------------------------------------------
constexpr float kFp8Max = 448.0f;
constexpr float kLeastMax = 0x1p-100f;

__device__ __forceinline__ float finite_size(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

// A block's scale, by which its elements are divided.  x / scale comes out of the
// rounded inverse y by two corrections q += (x - q scale) y: the first leaves q within a
// step of the quotient, and the second rounds it correctly then (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990),
// as long as the remainder is exact: where the scale is small, x and scale are taken 2^64
// times as large, so that remainders of quotients from 2^-11 on stay normal.  (A product
// with the inverse alone is a step of float32 away, and of bfloat16 rows, whose quotients
// often stand halfway between two e4m3, one element in 500 came out a step of e4m3 away.)
struct BlockScale {
    float scale, up, divisor, inverse;

    // m / 448 as a product, as a division by a number is on tensors.
    __device__ __forceinline__ explicit BlockScale(float most) : scale(most * (1.0f / kFp8Max)) {
        up = scale < 0x1p-64f ? 0x1p64f : 1.0f;
        divisor = scale * up;
        inverse = 1.0f / divisor;
    }
    // At most 448 and a few steps, which are 448 in e4m3; NaN of what is not finite.
    __device__ __forceinline__ float quotient(float x) const {
        const float a = x * up;
        float q = a * inverse;
        q = __builtin_fmaf(__builtin_fmaf(-q, divisor, a), inverse, q);
        q = __builtin_fmaf(__builtin_fmaf(-q, divisor, a), inverse, q);
        return __builtin_copysignf(q, x);  // (of -0 as well)
    }
};

// Two e4m3 in bits 0..15 of a word (HI: 16..31 of `old`), rounded to nearest even.
template <bool HI>
__device__ __forceinline__ int pack_fp8(float a, float b, const BlockScale &s, int old) {
    return __builtin_amdgcn_cvt_pk_fp8_f32(s.quotient(a), s.quotient(b), old, HI);
}

__device__ __forceinline__ uint2 pack8_fp8(const float (&f)[8], const BlockScale &s) {
    const int lo = pack_fp8<true>(f[2], f[3], s, pack_fp8<false>(f[0], f[1], s, 0));
    const int hi = pack_fp8<true>(f[6], f[7], s, pack_fp8<false>(f[4], f[5], s, 0));
    return {static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}

__device__ __forceinline__ void store8_fp8(uint8_t *p, int have, uint2 v) {
    if (have >= 8) {
        typedef uint32_t any2 __attribute__((ext_vector_type(2), aligned(1)));
        *reinterpret_cast<any2 *>(p) = any2{v.x, v.y};
    } else {
        const uint64_t all = static_cast<uint64_t>(v.y) << 32 | v.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < have) p[i] = static_cast<uint8_t>(all >> (8 * i));
        }
    }
}

// Elements [at, at + 8) of a row of `width`, zeros behind its end, without a branch
// where the row has 16 bytes: they are read from before its end and moved.  NONE: zeros
// alone, read from the row's beginning.
enum Row : int { kNarrowRow = 0, kRaggedRow = 1, kWholeRow = 2 };  // less than 16 bytes; whole chunks of 8 elements

template <class T, int ROW>
__device__ __forceinline__ void load8(const T *row, int at, int width, bool none, float (&f)[8]) {
    constexpr int V = kVec<T>;
    if constexpr (ROW == kNarrowRow) {
        load_some<T, 8>(row + at, none ? 0 : width - at, f);
    } else {
#pragma unroll
        for (int k = 0; k < 8; k += V) {
            const int to = at + k;
            const int from = none ? 0 : to < width - V ? to : width - V;
            auto raw = load16(reinterpret_cast<const char *>(row + from));
            if constexpr (ROW == kRaggedRow) {
                raw = cut<T>(raw, to, none ? 0 : width);
            } else if (none || to >= width) {
                raw = i32x4{0, 0, 0, 0};
            }
            union {
                i32x4 all;
                T e[V];
            } u{raw};
#pragma unroll
            for (int i = 0; i < V; ++i) f[k + i] = static_cast<float>(u.e[i]);
        }
    }
}

// 16 lanes a block, 8 elements each; a workgroup takes the same blocks of 16
// rows, whose scales stand side by side.  The grid's x runs over groups of
// kQuantizeBlocks blocks of a row, y over the rows.  (32768 x 2048 bfloat16: 36.6 us, 37.3
// with one block, 38.7 with four; gated 58.2 with one, 62.9 with two.)
template <bool GATE>
constexpr int kQuantizeBlocks = GATE ? 1 : 2;

template <class T, int ACT, bool GATE, int ROW>
__global__ __launch_bounds__(kGateBlock) void quantize_rows_kernel(const GateWork w) {
    const RowSpan live = live_rows(w.offsets, w.experts, static_cast<int>(w.num_rows));
    constexpr int kBlocks = kQuantizeBlocks<GATE>;
    const int g = threadIdx.x & 15, first = blockIdx.x * kBlocks;
    for (size_t r = static_cast<size_t>(blockIdx.y) * 16 + threadIdx.x / 16; r < w.num_rows;
         r += static_cast<size_t>(gridDim.y) * 16) {
        const int row = static_cast<int>(r);
        const bool has = row >= live.lo && row < live.hi;
        if (!has && !w.clear) continue;
        const T *in = static_cast<const T *>(w.rows) + r * w.rows_stride;
        float f[kBlocks][8], b[kBlocks][8];
        if (has) {
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                const int c = (first + j) * kScaleBlock + 8 * g;
                load8<T, ROW>(in, c, w.width, false, f[j]);
                if constexpr (GATE) load8<T, ROW>(in + w.width, c, w.width, false, b[j]);
            }
        } else {  // (is not read)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[j][i] = b[j][i] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int c = (first + j) * kScaleBlock + 8 * g, have = w.width - c;
            float most = kLeastMax;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (GATE) f[j][i] = activate<ACT, std::is_same_v<T, float>>(f[j][i]).value * b[j][i];
                most = __builtin_fmaxf(most, finite_size(f[j][i]));
            }
            most = group_max<16>(most);
            const BlockScale scale(most);
            const uint2 v = pack8_fp8(f[j], scale);
            if (have > 0) {
                store8_fp8(static_cast<uint8_t *>(w.out) + r * w.out_stride + c, have, v);
                if (g == 0) w.scales[static_cast<size_t>(first + j) * w.num_rows + r] = scale.scale;
            }
        }
    }
}

// 128 x 128 elements of a matrix a workgroup: 16 lanes a row, 16 rows a step.
struct QuantizeWeightsWork {
    const void *in;
    uint8_t *out;   // (experts, rows, width), contiguous
    float *scales;  // (experts, blocks of rows, blocks of width)
    size_t in_stride, in_expert;
    int experts, rows, width;
};

template <class T, int ROW>
__global__ __launch_bounds__(kGateBlock) void quantize_weights_kernel(const QuantizeWeightsWork w) {
    __shared__ float found[kGateBlock / 64];
    const int g = threadIdx.x & 15, sub = threadIdx.x / 16;
    const size_t across = (w.width + kScaleBlock - 1) / kScaleBlock, down = (w.rows + kScaleBlock - 1) / kScaleBlock;
    for (size_t job = blockIdx.x; job < across * down * w.experts; job += gridDim.x) {
        const int c = static_cast<int>(job % across) * kScaleBlock + 8 * g;
        const int r0 = static_cast<int>(job / across % down) * kScaleBlock;
        const size_t e = job / (across * down);
        const T *in = static_cast<const T *>(w.in) + e * w.in_expert;
        float f[8][8];
        float most = kLeastMax;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = r0 + 16 * j + sub;
            load8<T, ROW>(in + static_cast<size_t>(r < w.rows ? r : w.rows - 1) * w.in_stride, c, w.width, r >= w.rows, f[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) most = __builtin_fmaxf(most, finite_size(f[j][i]));
        }
        most = group_max<64>(most);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) found[threadIdx.x / 64] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kGateBlock / 64; ++i) most = __builtin_fmaxf(most, found[i]);
        const BlockScale scale(most);
        if (threadIdx.x == 0) w.scales[job] = scale.scale;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = r0 + 16 * j + sub;
            if (r < w.rows && c < w.width) {
                store8_fp8(w.out + (e * w.rows + r) * w.width + c, w.width - c, pack8_fp8(f[j], scale));
            }
        }
    }
}

}  // namespace rs
