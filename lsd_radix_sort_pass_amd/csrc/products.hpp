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
    unsigned jobs;   // tiles at most (of the square ones, which workgroups take in turn)
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
// Which tile a workgroup takes.  Consecutive workgroups go to the eight XCDs in
// turn, each with an L2 of its own: XCD x takes tiles that stand together.  Within an
// expert they go over kTurn tiles of q, then p, so that the 32 workgroups of an XCD share
// both operands.
// ---------------------------------------------------------------------------
constexpr int kXcds = 8;
constexpr int kTurn = 4;

struct ResultTile {
    int expert;  // -1: none; `experts`: rows of no expert
    int q, p;    // tiles
    RowSpan rows;
};

__device__ __forceinline__ void within(int local, int q_tiles, int p_tiles, ResultTile &t) {
    const int turn = local / (kTurn * p_tiles), left = q_tiles - turn * kTurn, r = local - turn * kTurn * p_tiles;
    const int deep = left < kTurn ? left : kTurn;
    t.q = turn * kTurn + r % deep;
    t.p = r / deep;
}

// Of ragged rows: workgroup b's.  Every wave finds it by itself.  The tiles of rows of no
// expert, which take no time to speak of, are shared out after the others.
__device__ inline ResultTile rows_tile(const int32_t *offsets, int experts, int num_rows, int height, int p_tiles,
                                      bool clear, unsigned b) {
    ResultTile t{-1, 0, 0, {0, num_rows}};
    const int lane = threadIdx.x & 63;
    const unsigned xcd = b % kXcds;
    unsigned at = b / kXcds, job = 0;
    // Whether the workgroup's place on its XCD is within the share of `tiles` times
    // p_tiles jobs; then `job` is its own, or there is none left (past).
    bool past = false;
    const auto takes = [&](int tiles) {
        const unsigned jobs = static_cast<unsigned>(tiles) * static_cast<unsigned>(p_tiles);
        const unsigned chunk = (jobs + kXcds - 1) / kXcds;
        if (at >= chunk) {
            at -= chunk;
            return false;
        }
        job = xcd * chunk + at;
        past = job >= jobs;
        return !past;
    };
    if (offsets == nullptr) {
        const int all = tiles_of(num_rows, height);
        if (takes(all)) {
            t.expert = 0;
            within(static_cast<int>(job), all, p_tiles, t);
        }
        return t;
    }
    // Rows and tiles of up to 64 experts, a lane each, and the tiles up to it.
    RowSpan r{0, 0};
    int tiles = 0, upto = 0, all = 0;
    const auto look = [&](int base) {
        r = rows_of(offsets, base + lane < experts ? base + lane : experts - 1, num_rows);
        tiles = base + lane < experts ? tiles_of(r.hi - r.lo, height) : 0;
        upto = wave_prefix(tiles, lane);
        return __builtin_amdgcn_readlane(upto, 63);
    };
    for (int base = 0; base < experts; base += 64) all += look(base);
    if (takes(all)) {
        const int tile = static_cast<int>(job / static_cast<unsigned>(p_tiles));
        int gone = 0;
        for (int base = 0; base < experts; base += 64) {
            const int sum = experts <= 64 ? all : look(base);  // (up to 64: they are there)
            if (tile - gone < sum) {
                const int found = __ffsll(static_cast<unsigned long long>(__ballot(upto > tile - gone))) - 1;
                const int first = gone + __builtin_amdgcn_readlane(upto - tiles, found);
                t.expert = base + found;
                t.rows = {__builtin_amdgcn_readlane(r.lo, found), __builtin_amdgcn_readlane(r.hi, found)};
                within(static_cast<int>(job - static_cast<unsigned>(first) * static_cast<unsigned>(p_tiles)),
                       __builtin_amdgcn_readlane(tiles, found), p_tiles, t);
                return t;
            }
            gone += sum;
        }
        return t;
    }
    if (past || !clear) return t;
    const int before = row_bound(offsets, 0, num_rows);
    int from = row_bound(offsets, experts, num_rows);
    from = from < before ? before : from;
    const int rest = tiles_of(before + (num_rows - from), height);
    if (takes(rest)) {
        t.expert = experts;
        t.rows = {before, from};
        within(static_cast<int>(job), rest, p_tiles, t);
    }
    return t;
}

// Of the weights' gradient: every expert has the same tiles.
__device__ inline ResultTile weights_tile(int experts, int q_tiles, int p_tiles, unsigned b) {
    ResultTile t{-1, 0, 0, {0, 0}};
    const unsigned tiles = static_cast<unsigned>(q_tiles) * static_cast<unsigned>(p_tiles);
    const unsigned chunk = (tiles + kXcds - 1) / kXcds, e = b / (chunk * kXcds), local = b % (chunk * kXcds);
    const unsigned job = local % kXcds * chunk + local / kXcds;
    if (e >= static_cast<unsigned>(experts) || job >= tiles) return t;
    t.expert = static_cast<int>(e);
    within(static_cast<int>(job), q_tiles, p_tiles, t);
    return t;
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

// Eight e4m3 in float16, which holds each of them exactly.
__device__ __forceinline__ f16x8 from_fp8(int lo, int hi) {
    const auto two = [](int v, auto high) {
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, decltype(high)::value);
    };
    const auto a = __builtin_shufflevector(two(lo, std::false_type{}), two(lo, std::true_type{}), 0, 1, 2, 3);
    const auto b = __builtin_shufflevector(two(hi, std::false_type{}), two(hi, std::true_type{}), 0, 1, 2, 3);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Whether sums of products of 8-bit operands are taken whole, in float32: by the 16-bit
// instruction.  The 8-bit one takes half of its time, but keeps of a product only what
// stands at most 18 digits below the largest of the 128, and so loses up to 2^-11 of that one
// (measured 2^-11.5), some 3 10^-4 of a result: a quarter of what rounding to bfloat16 may take from
// it (the error in norm is 0.0017 either way), but more than rounding to float16 or float32.
template <class OUT>
constexpr bool kWhole8 = !std::is_same_v<OUT, bf16>;

// 128 elements of c in e4m3, 32 bytes a lane.  (The 8-bit instruction's own scales are 1.)
template <bool WHOLE>
__device__ __forceinline__ f32x4 mma16_fp8(i32x4 p0, i32x4 p1, i32x4 q0, i32x4 q1) {
    f32x4 c{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (WHOLE) {
        // (Which elements of c meet in an instruction is free, as long as both operands agree.)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(from_fp8(p0[0], p0[1]), from_fp8(q0[0], q0[1]), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(from_fp8(p0[2], p0[3]), from_fp8(q0[2], q0[3]), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(from_fp8(p1[0], p1[1]), from_fp8(q1[0], q1[1]), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(from_fp8(p1[2], p1[3]), from_fp8(q1[2], q1[3]), c, 0, 0, 0);
    }
    const i32x8 p = __builtin_shufflevector(p0, p1, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 q = __builtin_shufflevector(q0, q1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, c, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
}

// 32 x 32 results, 16 elements of c: lane l holds row l % 32 of an operand and its
// 16-byte chunk l / 32; the result's lane l holds column q = l % 32 and in element
// i the row p = 8 (i / 4) + 4 (l / 32) + i % 4.
template <class T>
__device__ __forceinline__ f32x16 mma32(i32x4 p, i32x4 q, f32x16 c) {
    if constexpr (std::is_same_v<T, bf16>) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0,
                                                       0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0, 0,
                                                      0);
    }
}

// ---------------------------------------------------------------------------
// Tiles of an operand in LDS
// ---------------------------------------------------------------------------
// A tile holds 128 bytes of c for each of SIDE rows (along), or the elements of SIDE
// columns for as many steps of c (across).  Its 16-byte chunks are exchanged so that
// the lanes that LDS serves at once (256 bytes, all 64 banks) meet every bank once.
template <class T>
constexpr int kStep = 128 / static_cast<int>(sizeof(T));  // elements of c in a tile

template <class T, int SIDE, bool ACROSS>
constexpr int kChunksPerRow = ACROSS ? SIDE * static_cast<int>(sizeof(T)) / 16 : 8;

// Byte address in a tile of 16-byte chunk `chunk` of row `row`.
template <class T, int SIDE, bool ACROSS>
__device__ __forceinline__ int tile_at(int row, int chunk) {
    const int turn = !ACROSS ? row >> 1 & 7
        : sizeof(T) == 4     ? (row >> 2 & 3) << 2
        : SIDE == 64         ? (row >> 1 & 1) << 2
                             : (row & 3) << 2;
    return row * (kChunksPerRow<T, SIDE, ACROSS> * 16) + ((chunk ^ turn) << 4);
}

// What a lane feeds into the matrix instructions of a tile for rows (along) or columns
// (across) mn and those behind it: in 16 bits 32 of them, one of four steps; else 16,
// one of two halves.
template <class T, int SIDE, bool ACROSS>
__device__ __forceinline__ i32x4 fragment(const char *tile, int mn, int part, int lane) {
    if constexpr (sizeof(T) == 2 && !ACROSS) {
        return *reinterpret_cast<const i32x4 *>(tile + tile_at<T, SIDE, false>(mn + (lane & 31), 2 * part + (lane >> 5)));
    } else if constexpr (sizeof(T) == 2) {
        // Two reads that turn 4 rows of 16 elements into 4 elements of each column.
        const int i = lane & 15, g = lane >> 4;
        union {
            s16x4 half[2];
            i32x4 all;
        } f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 16 * part + 8 * (g >> 1) + 4 * h + (i >> 2), col = mn + 16 * (g & 1);
            const char *at = tile + tile_at<T, SIDE, true>(row, (col >> 3) + (i >> 1 & 1)) + (i & 1) * 8;
            f.half[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(at));
        }
        return f.all;
    } else if constexpr (!ACROSS) {
        return *reinterpret_cast<const i32x4 *>(tile + tile_at<T, SIDE, false>(mn + (lane & 15), (lane >> 4) + 4 * part));
    } else {
        const int col = mn + (lane & 15);
        i32x4 f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 4 * ((lane >> 4) + 4 * part) + j;
            f[j] = *reinterpret_cast<const int *>(tile + tile_at<T, SIDE, true>(row, col >> 2) + (col & 3) * 4);
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
// operands of any alignment, width and stride, by THREADS of them.  The loads are clamped
// into range, without a branch between them, and what they should not have read is
// cleared before it is stored.  NARROW: rows of less than 16 bytes, element by element.
template <class T, int SIDE, bool ACROSS, bool NARROW, int THREADS = 256>
struct Staging {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    static constexpr int kChunks = kChunksPerRow<T, SIDE, ACROSS>;
    static constexpr int kLoads = SIDE * 8 / THREADS;
    const T *from[kLoads];  // along: the row; across: the column
    size_t stride;
    int rows, width, first;  // of the operand's matrix, and the tile's first row (along) or column (across)

    __device__ __forceinline__ void set(const T *base, size_t stride_, int rows_, int width_, int first_, int tid) {
        stride = stride_, rows = rows_, width = width_, first = first_;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + tid;
            if constexpr (ACROSS) {
                const int c = first + id % kChunks * V;
                from[i] = base + (NARROW ? 0 : c < width - V ? c : width - V);
            } else {
                const int r = first + id / kChunks;
                from[i] = base + static_cast<size_t>(r < rows ? r : rows - 1) * stride;
            }
        }
    }

    // The chunks of the step that begins at c.
    __device__ __forceinline__ void load(i32x4 (&raw)[kLoads], int c, int tid) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + tid;
            const T *p = from[i];
            int at = ACROSS ? first + id % kChunks * V : c + id % kChunks * V;
            if constexpr (ACROSS) {
                const int r = c + id / kChunks;
                p += static_cast<size_t>(r < rows ? r : rows - 1) * stride;
            } else if constexpr (!NARROW) {
                p += at < width - V ? at : width - V;
            }
            if constexpr (NARROW) {
                union {
                    T e[V];
                    i32x4 all;
                } u;
                u.all = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (at + j < width) u.e[j] = p[at + j];
                }
                raw[i] = u.all;
            } else {
                raw[i] = load16(reinterpret_cast<const char *>(p));
            }
        }
    }

    __device__ __forceinline__ void store(i32x4 (&raw)[kLoads], char *tile, int c, int tid) const {
        const bool whole = ACROSS ? first + SIDE <= width && c + kStep<T> <= rows : c + kStep<T> <= width;
        if (!whole) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int id = i * THREADS + tid;
                if constexpr (!NARROW) raw[i] = cut<T>(raw[i], (ACROSS ? first : c) + id % kChunks * V, width);
                // (Rows of the other kind hold results of their own, which are not stored.)
                if (ACROSS && c + id / kChunks >= rows) raw[i] = i32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int id = i * THREADS + tid;
            *reinterpret_cast<i32x4 *>(tile + tile_at<T, SIDE, ACROSS>(id / kChunks, id % kChunks)) = raw[i];
        }
    }
};

// ---------------------------------------------------------------------------
// Waits for this wave's reads and writes of LDS and for the other waves, but not
// for loads from memory on their way to registers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void lds_barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
    __builtin_amdgcn_s_barrier();
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" ::: "memory");
#endif
}

// Orders what lanes of a wave have written to LDS before what others of it read, and what
// they have read before what is written over it.  The LDS serves a wave's accesses in
// order: this costs no instruction, and keeps the compiler from moving one lane's access
// over another's, whose address it can show to differ.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ---------------------------------------------------------------------------
// Zeros in `height` rows of no expert (fewer at their end), `columns` of them from col on,
// by all of the workgroup's threads, 16 bytes a thread.
// ---------------------------------------------------------------------------
template <class OUT>
__device__ __forceinline__ void clear_tile(OUT *out, size_t stride, int width, RowTile t, int height, int num_rows,
                                           int col, int columns) {
    constexpr int V = kVec<OUT>;
    const int rest = t.rows.lo + (num_rows - t.rows.hi), first = t.tile * height;
    const int rows = rest - first < height ? rest - first : height, chunks = columns / V;
    const float zeros[V] = {};
    for (int i = threadIdx.x; i < rows * chunks; i += blockDim.x) {
        const int c = col + i % chunks * V;
        int r = first + i / chunks;
        r = r < t.rows.lo ? r : r - t.rows.lo + t.rows.hi;
        if (c < width) store_some<OUT, V>(out + static_cast<size_t>(r) * stride + c, width - c, zeros);
    }
}

// ---------------------------------------------------------------------------
// A wave's results to rows: from its own part of LDS, which holds rows of 64 results of
// 16 bits, their chunks exchanged, so that 8 lanes write 128 bytes of a row.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int result_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

template <class OUT>
__device__ __forceinline__ void rows_from_lds(const char *mine, OUT *out, size_t stride, int height, int q_first,
                                              int q_rows, int p_first, int pn, int lane) {
#pragma unroll 4
    for (int k = 0; k < height / 8; ++k) {
        const int row = 8 * k + (lane >> 3), chunk = lane & 7;
        const i32x4 v = *reinterpret_cast<const i32x4 *>(mine + result_at(row, chunk));
        const int qi = q_first + row, pi = p_first + 8 * chunk, have = pn - pi;
        if (qi >= q_rows || have <= 0) continue;
        OUT *to = out + static_cast<size_t>(qi) * stride + pi;
        if (have >= 8) {
            *reinterpret_cast<i32x4_any *>(to) = v;
        } else {
            union {
                i32x4 all;
                OUT e[8];
            } u{v};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e < have) to[e] = u.e[e];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The product of any sizes, alignments and strides: SIDE x SIDE results a workgroup of
// four waves, a quarter each; the loads of the next AHEAD steps are in flight while the
// present one is multiplied.  Two take less time where rows begin at 16 bytes (1024 rows
// 4096 x 4096 bfloat16 55 us, 69 with one), but more where they do not, as the 32 KiB cache
// has to hold the lines that two steps share (4003 rows of 7 experts 1001 x 1537 float16 47 us,
// 39 with one; steps of 256 bytes 45; loads of the whole 16-byte words that hold them 65).
// SIDE is 128 in 16 and 8 bits; in 32 bits, where the matrix instructions take eight
// times as long, 64 fills the CUs more evenly: the gradients of 4093 rows of 8 experts
// 515 x 1030 112 us, 169 with 128.
// ---------------------------------------------------------------------------
template <class T>
constexpr int kSquare = sizeof(T) == 4 ? 64 : 128;

template <class T, class OUT, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS, int AHEAD, bool NARROW>
__global__ __launch_bounds__(256, kSquare<T> == 64 ? 4 : sizeof(T) == 1 ? 2 : 4 - AHEAD) void product_kernel(const ProductWork<T, OUT> w) {
    constexpr bool kFp8 = std::is_same_v<T, fp8>;
    constexpr int SIDE = kSquare<T>, kHalf = SIDE / 2;
    __shared__ __align__(16) char both_tiles[2 * SIDE * 128];
    char *const q_tile = both_tiles, *const p_tile = both_tiles + SIDE * 128;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q_wave = (wave >> 1) * kHalf, p_wave = (wave & 1) * kHalf;
    const int num_rows = static_cast<int>(w.num_rows);

    const int p_tiles = (w.pn + SIDE - 1) / SIDE, q_tiles = (w.qn + SIDE - 1) / SIDE;
    for (unsigned job = blockIdx.x; job < w.jobs; job += gridDim.x) {
        const ResultTile t = RAGGED_C ? weights_tile(w.experts, q_tiles, p_tiles, job)
                                      : rows_tile(w.offsets, w.experts, num_rows, SIDE, p_tiles, w.clear, job);
        if (t.expert < 0) continue;
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
                continue;
            }
            q_rows = t.rows.hi - t.rows.lo;
            c_n = w.cn;
            first_row = t.rows.lo;
            q += static_cast<size_t>(first_row) * w.q_stride;
            out += static_cast<size_t>(first_row) * w.out_stride;
            p += static_cast<size_t>(expert) * w.p_expert;
        }
        if (static_cast<unsigned>(q0) >= static_cast<unsigned>(q_rows) || p0 >= w.pn) continue;

        // In 16 bits 32 x 32 results an instruction, else 16 x 16.
        constexpr int kSide = sizeof(T) == 2 ? 32 : 16, kCount = kHalf / kSide;
        using Acc = std::conditional_t<sizeof(T) == 2, f32x16, f32x4>;
        Acc acc[kCount][kCount];
#pragma unroll
        for (auto &a : acc) {
#pragma unroll
            for (auto &b : a) b = Acc{};
        }
        Staging<T, SIDE, Q_ACROSS, NARROW> sq;
        Staging<T, SIDE, P_ACROSS, NARROW> sp;
        i32x4 raw_q[AHEAD][SIDE / 32], raw_p[AHEAD][SIDE / 32];
        // (What lies behind the end is loaded from before it, and not used: a load in a
        // branch would have to be waited for before the next.)
        const auto load = [&](int c, auto set) __attribute__((always_inline)) {
            sq.load(raw_q[decltype(set)::value], c, tid);
            sp.load(raw_p[decltype(set)::value], c, tid);
        };
        const auto step = [&](int c, auto set) __attribute__((always_inline)) {
            lds_barrier();
            sq.store(raw_q[decltype(set)::value], q_tile, c, tid);
            sp.store(raw_p[decltype(set)::value], p_tile, c, tid);
            lds_barrier();
            [[maybe_unused]] float scale[kCount], matrix_scale = 1.0f;
            if constexpr (kFp8) {  // (before the loads that nothing waits for yet)
                const int block = c / kScaleBlock, blocks = (w.cn + kScaleBlock - 1) / kScaleBlock;
                const int p_blocks = (w.pn + kScaleBlock - 1) / kScaleBlock;
                const float ps = w.p_scales[(static_cast<size_t>(expert) * p_blocks + p0 / kScaleBlock) * blocks + block];
                // (Whole sums are multiplied by both in turn, which leaves the compiler the registers for
                // products beside the conversions: 2150 us, 2530 by the scales' product.)
                if constexpr (kWhole8<OUT>) matrix_scale = ps;
#pragma unroll
                for (int j = 0; j < kCount; ++j) {
                    int r = q0 + q_wave + 16 * j + (lane & 15);
                    r = r < q_rows ? r : q_rows - 1;
                    scale[j] = w.q_scales[block * w.num_rows + first_row + r] * (kWhole8<OUT> ? 1.0f : ps);
                }
            }
            load(c + AHEAD * kStep<T>, set);
            if constexpr (kFp8) {
                i32x4 fp[kCount][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < kCount; ++i) fp[i][h] = fragment<T, SIDE, false>(p_tile, p_wave + 16 * i, h, lane);
                }
#pragma unroll
                for (int j = 0; j < kCount; ++j) {
                    const i32x4 fq0 = fragment<T, SIDE, false>(q_tile, q_wave + 16 * j, 0, lane);
                    const i32x4 fq1 = fragment<T, SIDE, false>(q_tile, q_wave + 16 * j, 1, lane);
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
                        const f32x4 part = mma16_fp8<kWhole8<OUT>>(fp[i][0], fp[i][1], fq0, fq1);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float sum = kWhole8<OUT> ? part[r] * scale[j] : part[r];
                            acc[i][j][r] = __builtin_fmaf(sum, kWhole8<OUT> ? matrix_scale : scale[j], acc[i][j][r]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < (sizeof(T) == 2 ? 4 : 2); ++k) {
                    i32x4 fp[kCount], fq[kCount];
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
                        fp[i] = fragment<T, SIDE, P_ACROSS>(p_tile, p_wave + kSide * i, k, lane);
                        fq[i] = fragment<T, SIDE, Q_ACROSS>(q_tile, q_wave + kSide * i, k, lane);
                    }
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
#pragma unroll
                        for (int j = 0; j < kCount; ++j) {
                            if constexpr (sizeof(T) == 2) {
                                acc[i][j] = mma32<T>(fp[i], fq[j], acc[i][j]);
                            } else {
                                acc[i][j] = mma16<T>(fp[i], fq[j], acc[i][j]);
                            }
                        }
                    }
                }
            }
        };
        if (c_n > 0) {
            sq.set(q, w.q_stride, Q_ACROSS ? c_n : q_rows, Q_ACROSS ? w.qn : c_n, q0, tid);
            sp.set(p, w.p_stride, P_ACROSS ? c_n : w.pn, P_ACROSS ? w.pn : c_n, p0, tid);
            constexpr std::integral_constant<int, 0> first{};
            constexpr std::integral_constant<int, AHEAD - 1> second{};
            load(0, first);
            if constexpr (AHEAD == 2) load(kStep<T>, second);
#pragma nounroll
            for (int c = 0; c < c_n; c += AHEAD * kStep<T>) {
                step(c, first);
                if constexpr (AHEAD == 2) {
                    if (c + kStep<T> < c_n) step(c + kStep<T>, second);
                }
            }
        }
        if constexpr (sizeof(OUT) == 2) {
            lds_barrier();  // (the tiles have been read)
            char *mine = both_tiles + wave * 8192;
            typedef OUT t4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int j = 0; j < kCount; ++j) {
                const int row = kSide * j + lane % kSide;
#pragma unroll
                for (int i = 0; i < kCount; ++i) {
#pragma unroll
                    for (int a = 0; a < (sizeof(T) == 2 ? 4 : 1); ++a) {
                        t4 v;
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = static_cast<OUT>(acc[i][j][4 * a + r]);
                        const int p = kSide * i + 8 * a + 4 * (lane / kSide);
                        *reinterpret_cast<t4 *>(mine + result_at(row, p / 8) + p % 8 * 2) = v;
                    }
                }
            }
            wave_exchange();
            rows_from_lds(mine, out, w.out_stride, 64, q0 + q_wave, q_rows, p0 + p_wave, w.pn, lane);
            continue;
        }
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int qi = q0 + q_wave + kSide * j + lane % kSide;
            if (qi >= q_rows) continue;
            OUT *row = out + static_cast<size_t>(qi) * w.out_stride;
#pragma unroll
            for (int i = 0; i < kCount; ++i) {
#pragma unroll
                for (int a = 0; a < (sizeof(T) == 2 ? 4 : 1); ++a) {
                    const int pi = p0 + p_wave + kSide * i + 8 * a + 4 * (lane / kSide);
                    float f[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) f[r] = acc[i][j][4 * a + r];
                    if (pi < w.pn) store_some<OUT, 4>(row + pi, w.pn - pi, f);
                }
            }
        }
    }
}

}  // namespace rs
