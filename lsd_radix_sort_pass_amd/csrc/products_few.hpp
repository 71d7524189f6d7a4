// products_few.hpp -- the experts' products for few rows an expert, as in decoding:
// the weights are read once and used for so few rows that memory bounds the product.
//
// A workgroup takes 16 * STRIPS output channels of an expert and up to 16 * ROWS of
// its rows.  Its waves share the contraction, 128 bytes of it a step in turn, so
// that they read adjacent parts of each weight row together, straight into the
// registers that the matrix instruction reads: no weight is used twice in a workgroup.
// In the end the waves' sums are joined in LDS, in the order of the waves.
#pragma once

#include "products.hpp"

namespace rs {

constexpr int kFewAhead = 4;  // steps whose loads are in flight together

// The 16 bytes of a row at element `at`, zeros behind `width`.  WHOLE: they exist.
template <class T, bool WHOLE>
__device__ __forceinline__ i32x4 row_chunk(const T *row, int at, int width) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if constexpr (WHOLE) return load16(reinterpret_cast<const char *>(row + at));
    const int from = at < width - V ? at : width - V;
    return cut<T>(load16(reinterpret_cast<const char *>(row + from)), at, width);
}

template <class T, class OUT, int WAVES, int STRIPS, int ROWS>
__global__ __launch_bounds__(64 * WAVES) void few_rows_kernel(const ProductWork<T, OUT> w) {
    constexpr bool kFp8 = std::is_same_v<T, fp8>;
    constexpr int V = 16 / static_cast<int>(sizeof(T)), kStepC = 8 * V;
    __shared__ __align__(16) f32x4 sums[WAVES - 1][STRIPS * ROWS][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int num_rows = static_cast<int>(w.num_rows), c_n = w.cn;
    constexpr int kCols = 16 * STRIPS, kHeight = 16 * ROWS;
    const unsigned p_tiles = static_cast<unsigned>((w.pn + kCols - 1) / kCols);
    const int p0 = static_cast<int>(blockIdx.x % p_tiles) * kCols;
    const RowTile t = find_tile(w.offsets, w.experts, num_rows, kHeight, static_cast<int>(blockIdx.x / p_tiles));
    if (t.expert < 0) return;
    OUT *out = w.out;
    if (t.expert == w.experts) {
        if (w.clear) clear_tile(out, w.out_stride, w.pn, t, kHeight, num_rows, p0, kCols);
        return;
    }
    const int q0 = t.tile * kHeight, left = t.rows.hi - t.rows.lo - q0, first_row = t.rows.lo + q0;
    if (left <= 0) return;

    // Rows of results that do not exist are others' again.
    const T *qr[ROWS], *pr[STRIPS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        const int r = 16 * j + i < left ? 16 * j + i : left - 1;
        qr[j] = w.q + static_cast<size_t>(first_row + r) * w.q_stride;
    }
#pragma unroll
    for (int s = 0; s < STRIPS; ++s) {
        const int r = p0 + 16 * s + i < w.pn ? p0 + 16 * s + i : w.pn - 1;
        pr[s] = w.p + static_cast<size_t>(t.expert) * w.p_expert + static_cast<size_t>(r) * w.p_stride;
    }
    f32x4 acc[STRIPS][ROWS];
#pragma unroll
    for (auto &a : acc) {
#pragma unroll
        for (auto &b : a) b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // Scales: of the lane's rows, and of the strips' 128 x 128 block.
    const size_t blocks = (static_cast<size_t>(c_n) + kScaleBlock - 1) / kScaleBlock;
    const size_t p_blocks = (static_cast<size_t>(w.pn) + kScaleBlock - 1) / kScaleBlock;
    const float *ps = kFp8 ? w.p_scales + (static_cast<size_t>(t.expert) * p_blocks + p0 / kScaleBlock) * blocks : nullptr;

    // AHEAD steps from element c on, WAVES steps apart.
    const auto steps = [&](int c, auto ahead, auto whole) __attribute__((always_inline)) {
        constexpr int kAhead = decltype(ahead)::value;
        constexpr bool kWhole = decltype(whole)::value;
        i32x4 fp[kAhead][STRIPS][2], fq[kAhead][ROWS][2];
        float scale[kAhead][ROWS];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int at = c + a * WAVES * kStepC + g * V;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int s = 0; s < STRIPS; ++s) fp[a][s][h] = row_chunk<T, kWhole>(pr[s], at + 4 * V * h, c_n);
#pragma unroll
                for (int j = 0; j < ROWS; ++j) fq[a][j][h] = row_chunk<T, kWhole>(qr[j], at + 4 * V * h, c_n);
            }
            if constexpr (kFp8) {
                const int block = c / kScaleBlock + a * WAVES;
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    const int r = 16 * j + i < left ? 16 * j + i : left - 1;
                    scale[a][j] = w.q_scales[static_cast<size_t>(block) * w.num_rows + first_row + r] * ps[block];
                }
            }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
#pragma unroll
            for (int s = 0; s < STRIPS; ++s) {
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    if constexpr (kFp8) {
                        const f32x4 part = mma16_fp8<kWhole8<OUT>>(fp[a][s][0], fp[a][s][1], fq[a][j][0], fq[a][j][1]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            acc[s][j][r] = __builtin_fmaf(part[r], scale[a][j], acc[s][j][r]);
                        }
                    } else {
                        acc[s][j] = mma16<T>(fp[a][s][0], fq[a][j][0], acc[s][j]);
                        acc[s][j] = mma16<T>(fp[a][s][1], fq[a][j][1], acc[s][j]);
                    }
                }
            }
        }
    };
    // The workgroups of an XCD begin at different places: rows whose stride is a large
    // power of two stand in the same channel of its L2, and all would ask that one.
    constexpr int kSpan = WAVES * kStepC, kBatch = kFewAhead * kSpan;
    const int batches = c_n / kBatch;
    int batch = batches > 0 ? static_cast<int>(blockIdx.x / 8 % static_cast<unsigned>(batches)) : 0;
#pragma nounroll
    for (int b = 0; b < batches; ++b) {
        steps(batch * kBatch + wave * kStepC, std::integral_constant<int, kFewAhead>{}, std::true_type{});
        batch = batch + 1 < batches ? batch + 1 : 0;
    }
    int c = batches * kBatch + wave * kStepC;
#pragma nounroll
    for (; c + kStepC <= c_n; c += kSpan) steps(c, std::integral_constant<int, 1>{}, std::true_type{});
    if (c < c_n) steps(c, std::integral_constant<int, 1>{}, std::false_type{});

    if (wave > 0) {
#pragma unroll
        for (int s = 0; s < STRIPS; ++s) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) sums[wave - 1][s * ROWS + j][lane] = acc[s][j];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
#pragma unroll
        for (int s = 0; s < STRIPS; ++s) {
            f32x4 all = acc[s][j];
#pragma unroll
            for (int k = 0; k < WAVES - 1; ++k) all += sums[k][s * ROWS + j][lane];
            const int r = 16 * j + i, pi = p0 + 16 * s + 4 * g;
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = all[e];
            if (r < left && pi < w.pn) {
                store_some<OUT, 4>(out + static_cast<size_t>(first_row + r) * w.out_stride + pi, w.pn - pi, f);
            }
        }
    }
}

}  // namespace rs
