// products.hpp -- gfx950 kernels of the experts' matrix products: token rows
// that stand sorted by expert times each expert's weights, and the gradients.
//
// One form serves the three products:  C[q][p] = sum over c of Q[q, c] P[p, c],
//
//   forward          q a row of the expert, p an output channel, c an input channel
//   grad of rows     q a row,               p an input channel,  c an output channel
//   grad of weights  q an output channel,   p an input channel,  c a row
//
// where an operand stands in memory "along" c (consecutive elements differ in c)
// or "across" it (consecutive elements differ in q or p).  P is the matrix
// instruction's first operand, so that a lane ends with consecutive elements of
// one row of C.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "elements.hpp"

namespace rs {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

struct fp8 {  // e4m3, four to a word
    uint8_t bits;
};

constexpr int kScaleBlock = 128;  // elements that share a scale, along c and (of weights) along p

// What a product works on.  Rows stand expert by expert: expert e has the rows
// [offsets[e], offsets[e + 1]); without offsets the one expert has all.
template <class T, class OUT>
struct ProductWork {
    const T *q, *p;
    OUT *out;
    size_t q_stride, p_stride, out_stride;  // elements between rows
    size_t p_expert, out_expert;            // between experts' matrices (0: rows)
    const int32_t *offsets;
    const float *q_scales, *p_scales;  // 8 bits: [blocks of c][num_rows], [expert][blocks of p][blocks of c]
    size_t num_rows;
    int experts;
    int qn, pn, cn;  // widths; of the ragged one of qn and cn: 0
    bool clear;      // write zeros to the rows of no expert
};

// ---------------------------------------------------------------------------
// Rows of an expert, and tiles of them
// ---------------------------------------------------------------------------
struct RowSpan {
    int lo, hi;
};

// Offsets are taken into range, so that no value of theirs leads outside.
__device__ __forceinline__ int row_bound(const int32_t *offsets, int i, int num_rows) {
    const int v = offsets[i];
    return v < 0 ? 0 : v > num_rows ? num_rows : v;
}

__device__ __forceinline__ RowSpan rows_of(const int32_t *offsets, int e, int num_rows) {
    if (offsets == nullptr) return {0, num_rows};
    const int lo = row_bound(offsets, e, num_rows), hi = row_bound(offsets, e + 1, num_rows);
    return {lo, hi < lo ? lo : hi};
}

__device__ __forceinline__ int tiles_of(int rows, int height) {
    return static_cast<int>((static_cast<unsigned>(rows) + height - 1) / height);
}

// Sum of x over this lane and those before it.
__device__ __forceinline__ int wave_prefix(int x, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
    return x;
}

struct RowTile {
    int expert;  // `experts`: rows of no expert
    int tile;    // number of the tile within the expert's rows
    RowSpan rows;
};

// Tile t of the tiles of `height` rows, expert by expert, that all experts' rows
// make; behind them those of the rows of no expert: the ones before the first
// offset and behind the last, in this order (rows.lo counts the former,
// rows.hi the place where the latter begin).  expert -1: t lies behind all.
// Every wave finds it by itself, 64 experts at a time; all lanes must be active.
__device__ inline RowTile find_tile(const int32_t *offsets, int experts, int num_rows, int height, int t) {
    const int lane = threadIdx.x & 63;
    if (offsets == nullptr) {
        return {t < tiles_of(num_rows, height) ? 0 : -1, t, {0, num_rows}};
    }
    for (int base = 0; base < experts; base += 64) {
        const int e = base + lane < experts ? base + lane : experts - 1;
        const RowSpan r = rows_of(offsets, e, num_rows);
        const int tiles = base + lane < experts ? tiles_of(r.hi - r.lo, height) : 0;
        const int upto = wave_prefix(tiles, lane);
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (t < all) {
            const int at = __ffsll(static_cast<unsigned long long>(__ballot(upto > t))) - 1;
            return {base + at, t - __builtin_amdgcn_readlane(upto - tiles, at),
                    {__builtin_amdgcn_readlane(r.lo, at), __builtin_amdgcn_readlane(r.hi, at)}};
        }
        t -= all;
    }
    const int before = row_bound(offsets, 0, num_rows), end = row_bound(offsets, experts, num_rows);
    const int from = end < before ? before : end;
    return {t < tiles_of(before + (num_rows - from), height) ? experts : -1, t, {before, from}};
}

// ---------------------------------------------------------------------------
// Matrix instructions: 16 x 16 results, 16 bytes of c of each operand a lane.
// Lane l holds row l % 16 of an operand and its 16-byte chunk l / 16 of c; the
// result's lane l holds column q = l % 16 and rows p = 4 (l / 16) + 0..3.
// ---------------------------------------------------------------------------
template <class T>
__device__ __forceinline__ f32x4 mma16(i32x4 p, i32x4 q, f32x4 c) {
    if constexpr (std::is_same_v<T, bf16>) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0,
                                                       0, 0);
    } else if constexpr (std::is_same_v<T, f16>) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0, 0,
                                                      0);
    } else {
        static_assert(std::is_same_v<T, float>);
        const f32x4 a = __builtin_bit_cast(f32x4, p), b = __builtin_bit_cast(f32x4, q);
        // Which four elements of c meet in an instruction is free, as long as
        // both operands agree.
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
}

// 128 elements of c in e4m3, 32 bytes a lane; the instruction's own scales are 1.
__device__ __forceinline__ f32x4 mma16_fp8(i32x4 p0, i32x4 p1, i32x4 q0, i32x4 q1) {
    const i32x8 p = __builtin_shufflevector(p0, p1, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 q = __builtin_shufflevector(q0, q1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0x7F7F7F7F, 0,
                                                            0x7F7F7F7F);
}

// ---------------------------------------------------------------------------
// Tiles of an operand in LDS
// ---------------------------------------------------------------------------
// A tile holds 128 bytes of c for each of 128 rows (along), or the elements of
// 128 columns for as many steps of c as fill 16 KiB (across).  Its 16-byte
// chunks (along) and 32-byte units (across) are exchanged so that the 16 or 32 lanes
// that LDS serves at once (256 bytes, all 64 banks) meet every bank once.
constexpr int kTileBytes = 16384;

template <class T>
constexpr int kStep = 128 / static_cast<int>(sizeof(T));  // elements of c in a tile

// Byte address in a tile of 16-byte chunk `chunk` of row `row`.
template <class T, bool ACROSS>
__device__ __forceinline__ int tile_at(int row, int chunk) {
    if constexpr (!ACROSS) {
        return row * 128 + ((chunk ^ (row >> 1 & 7)) << 4);
    } else if constexpr (sizeof(T) == 2) {
        const int turn = (row & 3) | ((row >> 1) & 4);
        return row * 256 + ((chunk ^ (turn << 1)) << 4);
    } else {
        return row * 512 + ((chunk ^ ((row >> 2 & 3) << 2)) << 4);
    }
}

template <class T, bool ACROSS>
constexpr int kChunksPerRow = ACROSS ? 128 * static_cast<int>(sizeof(T)) / 16 : 8;

// The 16 bytes that lane `lane` feeds into the matrix instruction `half` (of 2)
// of rows (along) or columns (across) mn .. mn + 15 of a tile.
template <class T, bool ACROSS>
__device__ __forceinline__ i32x4 fragment(const char *tile, int mn, int half, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (!ACROSS) {
        return *reinterpret_cast<const i32x4 *>(tile + tile_at<T, false>(mn + i, g + 4 * half));
    } else if constexpr (sizeof(T) == 2) {
        // Two reads that turn 4 rows of 16 elements into 4 elements of each column.
        union {
            s16x4 part[2];
            i32x4 all;
        } f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 32 * half + 8 * g + 4 * h + (i >> 2);
            const char *at = tile + tile_at<T, true>(row, (mn >> 3) + (i >> 1 & 1)) + (i & 1) * 8;
            f.part[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(at));
        }
        return f.all;
    } else {
        i32x4 f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 4 * (g + 4 * half) + j, col = mn + i;
            f[j] = *reinterpret_cast<const int *>(tile + tile_at<T, true>(row, col >> 2) + (col & 3) * 4);
        }
        return f;
    }
}

// 16 bytes from any address.
__device__ __forceinline__ i32x4 load16(const char *p) { return *reinterpret_cast<const i32x4_any *>(p); }

// The elements [at, at + V) of a row of `width` elements as 16 bytes, zeros behind
// its end: `raw` are the V elements from min(at, width - V) on.
template <class T>
__device__ __forceinline__ i32x4 cut(i32x4 raw, int at, int width) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int over = at + V - width;
    if (over <= 0) return raw;
    if (over >= V) return i32x4{0, 0, 0, 0};
    const auto v = __builtin_bit_cast(unsigned __int128, raw) >> (over * 8 * static_cast<int>(sizeof(T)));
    return __builtin_bit_cast(i32x4, v);
}

// A tile's elements on their way from memory through registers to LDS, for
// operands of any alignment, width and stride.  256 threads, 4 chunks each; the
// loads are clamped into range, without a branch between them, and what they
// should not have read is cleared before it is stored.
template <class T, bool ACROSS>
struct Staging {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    static constexpr int kChunks = kChunksPerRow<T, ACROSS>;
    i32x4 raw[4];

    // rows: those of the operand's matrix that exist; width: elements of a row;
    // row0, col0: the tile's first.
    __device__ __forceinline__ void load(const T *base, size_t stride, int rows, int width, int row0, int col0, int tid) {
        if (width >= V) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int id = i * 256 + tid;
                int r = row0 + id / kChunks, c = col0 + id % kChunks * V;
                r = r < rows ? r : rows - 1;
                c = c < width - V ? c : width - V;
                raw[i] = load16(reinterpret_cast<const char *>(base + static_cast<size_t>(r) * stride + c));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int id = i * 256 + tid;
                int r = row0 + id / kChunks;
                const int c = col0 + id % kChunks * V;
                r = r < rows ? r : rows - 1;
                const T *row = base + static_cast<size_t>(r) * stride;
                union {
                    T e[V];
                    i32x4 all;
                } u;
                u.all = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (c + j < width) u.e[j] = row[c + j];
                }
                raw[i] = u.all;
            }
        }
    }

    __device__ __forceinline__ void store(char *tile, int rows, int width, int row0, int col0, int tid) {
        const bool whole = row0 + 1024 / kChunks <= rows && col0 + kChunks * V <= width;
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int id = i * 256 + tid, c = col0 + id % kChunks * V;
                if (width >= V) raw[i] = cut<T>(raw[i], c, width);
                // Rows of the other kind hold results of their own, which are not stored.
                if (ACROSS && row0 + id / kChunks >= rows) raw[i] = i32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = i * 256 + tid;
            *reinterpret_cast<i32x4 *>(tile + tile_at<T, ACROSS>(id / kChunks, id % kChunks)) = raw[i];
        }
    }
};

// ---------------------------------------------------------------------------
// Zeros in rows of no expert: 128 of them (fewer at their end), columns
// [col, col + 128).
// ---------------------------------------------------------------------------
template <class OUT>
__device__ __forceinline__ void clear_tile(OUT *out, size_t stride, int width, RowTile t, int height, int num_rows,
                                           int col, int columns) {
    const int rest = t.rows.lo + num_rows - t.rows.hi, first = t.tile * height;
    const int rows = rest - first < height ? rest - first : height;
    const int wide = width - col < columns ? width - col : columns;
    for (int i = threadIdx.x; i < rows * columns; i += blockDim.x) {
        const int c = i % columns;
        int r = first + i / columns;
        r = r < t.rows.lo ? r : r - t.rows.lo + t.rows.hi;
        if (c < wide) out[static_cast<size_t>(r) * stride + col + c] = OUT{};
    }
}

// ---------------------------------------------------------------------------
// The product of any sizes, alignments and strides: 128 x 128 results a
// workgroup of four waves, 64 x 64 a wave; the next tiles' loads are in flight
// while the present ones are multiplied.
// ---------------------------------------------------------------------------
template <class T, class OUT, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS>
__global__ __launch_bounds__(256, 2) void product_kernel(const ProductWork<T, OUT> w) {
    constexpr bool kFp8 = std::is_same_v<T, fp8>;
    __shared__ __align__(16) char q_tile[kTileBytes];
    __shared__ __align__(16) char p_tile[kTileBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int q_wave = (wave >> 1) * 64, p_wave = (wave & 1) * 64;
    const int num_rows = static_cast<int>(w.num_rows);

    const unsigned p_tiles = static_cast<unsigned>((w.pn + 127) / 128);
    const unsigned q_tiles = RAGGED_C ? static_cast<unsigned>((w.qn + 127) / 128) : 0;
    for (size_t job = blockIdx.x;; job += gridDim.x) {
        const T *q = w.q, *p = w.p;
        OUT *out = w.out;
        int q0, q_rows, c_n, expert;
        const int p0 = static_cast<int>(job % p_tiles) * 128;
        int first_row = 0;
        if constexpr (RAGGED_C) {
            const size_t t = job / p_tiles, e = t / q_tiles;
            if (e >= static_cast<size_t>(w.experts)) break;
            expert = static_cast<int>(e);
            q0 = static_cast<int>(t % q_tiles) * 128;
            q_rows = w.qn;
            const RowSpan r = rows_of(w.offsets, expert, num_rows);
            c_n = r.hi - r.lo;
            q += static_cast<size_t>(r.lo) * w.q_stride;
            p += static_cast<size_t>(r.lo) * w.p_stride;
            out += e * w.out_expert;
        } else {
            const size_t t = job / p_tiles;
            if (t > 0x7FFFFFFFu) break;
            const RowTile f = find_tile(w.offsets, w.experts, num_rows, 128, static_cast<int>(t));
            if (f.expert < 0) break;
            expert = f.expert;
            if (expert == w.experts) {
                if (!w.clear) break;
                clear_tile(out, w.out_stride, w.pn, f, 128, num_rows, p0, 128);
                continue;
            }
            q0 = f.tile * 128;
            q_rows = f.rows.hi - f.rows.lo;
            c_n = w.cn;
            first_row = f.rows.lo;
            q += static_cast<size_t>(first_row) * w.q_stride;
            out += static_cast<size_t>(first_row) * w.out_stride;
            p += static_cast<size_t>(expert) * w.p_expert;
        }

        f32x4 acc[4][4];
#pragma unroll
        for (auto &a : acc) {
#pragma unroll
            for (auto &b : a) b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        Staging<T, Q_ACROSS> sq;
        Staging<T, P_ACROSS> sp;
        const int q_have = Q_ACROSS ? c_n : q_rows, q_width = Q_ACROSS ? w.qn : c_n;
        const int p_have = P_ACROSS ? c_n : w.pn, p_width = P_ACROSS ? w.pn : c_n;
        const auto load = [&](int c) {
            sq.load(q, w.q_stride, q_have, q_width, Q_ACROSS ? c : q0, Q_ACROSS ? q0 : c, tid);
            sp.load(p, w.p_stride, p_have, p_width, P_ACROSS ? c : p0, P_ACROSS ? p0 : c, tid);
        };
        if (c_n > 0) load(0);
        for (int c = 0; c < c_n; c += kStep<T>) {
            __syncthreads();
            sq.store(q_tile, q_have, q_width, Q_ACROSS ? c : q0, Q_ACROSS ? q0 : c, tid);
            sp.store(p_tile, p_have, p_width, P_ACROSS ? c : p0, P_ACROSS ? p0 : c, tid);
            __syncthreads();
            if (c + kStep<T> < c_n) load(c + kStep<T>);
            if constexpr (kFp8) {
                const int block = c / kScaleBlock, blocks = (w.cn + kScaleBlock - 1) / kScaleBlock;
                const int p_blocks = (w.pn + kScaleBlock - 1) / kScaleBlock;
                const float ps = w.p_scales[(static_cast<size_t>(expert) * p_blocks + p0 / kScaleBlock) * blocks + block];
                float scale[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    int r = q0 + q_wave + 16 * j + (lane & 15);
                    r = r < q_rows ? r : q_rows - 1;
                    scale[j] = ps * w.q_scales[block * w.num_rows + first_row + r];
                }
                i32x4 fp[4][2], fq[4][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fp[i][h] = fragment<T, false>(p_tile, p_wave + 16 * i, h, lane);
                        fq[i][h] = fragment<T, false>(q_tile, q_wave + 16 * i, h, lane);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 part = mma16_fp8(fp[i][0], fp[i][1], fq[j][0], fq[j][1]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(part[r], scale[j], acc[i][j][r]);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    i32x4 fp[4], fq[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fp[i] = fragment<T, P_ACROSS>(p_tile, p_wave + 16 * i, h, lane);
                        fq[i] = fragment<T, Q_ACROSS>(q_tile, q_wave + 16 * i, h, lane);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = mma16<T>(fp[i], fq[j], acc[i][j]);
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int qi = q0 + q_wave + 16 * j + (lane & 15);
            if (qi >= q_rows) continue;
            OUT *row = out + static_cast<size_t>(qi) * w.out_stride;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pi = p0 + p_wave + 16 * i + 4 * (lane >> 4);
                float f[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) f[r] = acc[i][j][r];
                if (pi < w.pn) store_some<OUT, 4>(row + pi, w.pn - pi, f);
            }
        }
    }
}

}  // namespace rs
