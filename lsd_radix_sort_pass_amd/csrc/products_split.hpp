// products_split.hpp -- the experts' products with few results and a long contraction,
// for whose square tiles there are too few: 64 x 64 results a workgroup of eight waves
// that share the contraction, 128 bytes of it a step in turn.
//
// A wave brings its own steps through registers to its own part of LDS, so that no wave
// waits for another before the end, where their sums are joined in LDS in the order of
// the waves.  Tiles of 64 x 64 read an operand twice as often as those of 128 x 128, and are
// bound by what a CU takes in (128 KiB a step in 1.4 to 1.75 us): they pay while the others
// leave CUs empty.  256 rows 4096 x 4096 bfloat16 20 us, 46 with square tiles; the weights'
// gradient of 8192 rows 1024 x 1024 34 us, 172 with wide ones.  In 16 and 8 bits.
#pragma once

#include "products.hpp"

namespace rs {

constexpr int kSplitSide = 64, kSplitWaves = 8;

template <class T, class OUT, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS>
__global__ __launch_bounds__(64 * kSplitWaves) void split_kernel(const ProductWork<T, OUT> w) {
    static_assert(sizeof(T) <= 2);
    constexpr bool kFp8 = std::is_same_v<T, fp8>;
    constexpr int SIDE = kSplitSide, kTile = SIDE * 128, kSpan = kSplitWaves * kStep<T>;
    __shared__ __align__(16) char parts[kSplitWaves][2 * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int num_rows = static_cast<int>(w.num_rows);
    char *const q_tile = parts[wave], *const p_tile = q_tile + kTile;
    const int p_tiles = (w.pn + SIDE - 1) / SIDE, q_tiles = (w.qn + SIDE - 1) / SIDE;
    const ResultTile t = RAGGED_C ? weights_tile(w.experts, q_tiles, p_tiles, blockIdx.x)
                                  : rows_tile(w.offsets, w.experts, num_rows, SIDE, p_tiles, w.clear, blockIdx.x);
    if (t.expert < 0) return;
    const int q0 = t.q * SIDE, p0 = t.p * SIDE, expert = t.expert;
    const T *q = w.q, *p = w.p;
    OUT *out = w.out;
    int q_rows, c_n, first_row = 0;
    if constexpr (RAGGED_C) {
        const RowSpan r = rows_of(w.offsets, expert, num_rows);
        q_rows = w.qn;
        c_n = r.hi - r.lo;
        q += static_cast<size_t>(r.lo) * w.q_stride;
        p += static_cast<size_t>(r.lo) * w.p_stride;
        out += static_cast<size_t>(expert) * w.out_expert;
    } else {
        if (expert == w.experts) {
            clear_tile(out, w.out_stride, w.pn, RowTile{expert, t.q, t.rows}, SIDE, num_rows, p0, SIDE);
            return;
        }
        q_rows = t.rows.hi - t.rows.lo;
        c_n = w.cn;
        first_row = t.rows.lo;
        q += static_cast<size_t>(first_row) * w.q_stride;
        out += static_cast<size_t>(first_row) * w.out_stride;
        p += static_cast<size_t>(expert) * w.p_expert;
    }
    if (static_cast<unsigned>(q0) >= static_cast<unsigned>(q_rows) || p0 >= w.pn) return;

    constexpr int kSide = sizeof(T) == 2 ? 32 : 16, kCount = SIDE / kSide;
    using Acc = std::conditional_t<sizeof(T) == 2, f32x16, f32x4>;
    Acc acc[kCount][kCount];
#pragma unroll
    for (auto &a : acc) {
#pragma unroll
        for (auto &b : a) b = Acc{};
    }
    if (c_n > 0) {
        Staging<T, SIDE, Q_ACROSS, false, 64> sq;
        Staging<T, SIDE, P_ACROSS, false, 64> sp;
        sq.set(q, w.q_stride, Q_ACROSS ? c_n : q_rows, Q_ACROSS ? w.qn : c_n, q0, lane);
        sp.set(p, w.p_stride, P_ACROSS ? c_n : w.pn, P_ACROSS ? w.pn : c_n, p0, lane);
        i32x4 raw_q[SIDE / 8], raw_p[SIDE / 8];
        sq.load(raw_q, wave * kStep<T>, lane);
        sp.load(raw_p, wave * kStep<T>, lane);
#pragma nounroll
        for (int c = wave * kStep<T>; c < c_n; c += kSpan) {
            sq.store(raw_q, q_tile, c, lane);
            sp.store(raw_p, p_tile, c, lane);
            wave_exchange();
            [[maybe_unused]] float scale[kCount];
            if constexpr (kFp8) {  // (before the loads that nothing waits for yet)
                const int block = c / kScaleBlock, blocks = (w.cn + kScaleBlock - 1) / kScaleBlock;
                const int p_blocks = (w.pn + kScaleBlock - 1) / kScaleBlock;
                const float ps =
                    w.p_scales[(static_cast<size_t>(expert) * p_blocks + p0 / kScaleBlock) * blocks + block];
#pragma unroll
                for (int j = 0; j < kCount; ++j) {
                    int r = q0 + 16 * j + (lane & 15);
                    r = r < q_rows ? r : q_rows - 1;
                    scale[j] = ps * w.q_scales[block * w.num_rows + first_row + r];
                }
            }
            sq.load(raw_q, c + kSpan, lane);  // (behind the end: from before it, not used)
            sp.load(raw_p, c + kSpan, lane);
            if constexpr (kFp8) {
                i32x4 fp[kCount][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < kCount; ++i) fp[i][h] = fragment<T, SIDE, false>(p_tile, 16 * i, h, lane);
                }
#pragma unroll
                for (int j = 0; j < kCount; ++j) {
                    const i32x4 fq0 = fragment<T, SIDE, false>(q_tile, 16 * j, 0, lane);
                    const i32x4 fq1 = fragment<T, SIDE, false>(q_tile, 16 * j, 1, lane);
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
                        const f32x4 part = mma16_fp8<kWhole8<OUT>>(fp[i][0], fp[i][1], fq0, fq1);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(part[r], scale[j], acc[i][j][r]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    i32x4 fp[kCount], fq[kCount];
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
                        fp[i] = fragment<T, SIDE, P_ACROSS>(p_tile, kSide * i, k, lane);
                        fq[i] = fragment<T, SIDE, Q_ACROSS>(q_tile, kSide * i, k, lane);
                    }
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
#pragma unroll
                        for (int j = 0; j < kCount; ++j) {
                            acc[i][j] = mma32<T>(fp[i], fq[j], acc[i][j]);
                        }
                    }
                }
            }
            wave_exchange();
        }
    }

    // The wave's sums to its part of LDS: 64 rows of 64, their chunks of four exchanged.
    const auto sum_at = [](int row, int chunk) { return row * (SIDE * 4) + ((chunk ^ (row & 15)) << 4); };
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
        const int row = kSide * j + lane % kSide;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
#pragma unroll
            for (int a = 0; a < (sizeof(T) == 2 ? 4 : 1); ++a) {
                f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * a + r];
                const int pi = kSide * i + 8 * a + 4 * (lane / kSide);
                *reinterpret_cast<f32x4 *>(q_tile + sum_at(row, pi / 4)) = v;
            }
        }
    }
    __syncthreads();
    const int row = static_cast<int>(threadIdx.x) / 8, at = static_cast<int>(threadIdx.x) % 8 * 2;
    const int pi = p0 + 4 * at;
    f32x4 all[2] = {};
#pragma unroll
    for (int k = 0; k < kSplitWaves; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) all[h] += *reinterpret_cast<const f32x4 *>(parts[k] + sum_at(row, at + h));
    }
    if (q0 + row < q_rows) {
        OUT *to = out + static_cast<size_t>(q0 + row) * w.out_stride + pi;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] = all[h][r];
            if (pi + 4 * h < w.pn) store_some<OUT, 4>(to + 4 * h, w.pn - pi - 4 * h, f);
        }
    }
}

}  // namespace rs
