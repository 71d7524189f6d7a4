// products_wide.hpp -- the experts' products in 16 bits for many rows an expert:
// 256 x 256 results a workgroup of eight waves, operands brought to LDS by the
// memory system itself, without passing through registers.
//
// The waves form two groups of four, one wave of each group on every SIMD.  Group
// g has the rows q = 128 g .. 128 g + 127, each of its waves 64 columns p, so a
// wave holds 128 x 64 results.  The contraction goes in stages of 64 bytes of c.
// In a slot, one group reads the operands of its next stage from LDS while the
// other multiplies; a barrier ends the slot and they change places.  A SIMD
// thus multiplies in every slot, and no wave has to hold two stages' operands.
// LDS is a ring of four stages, three of them on their way.
//
// A tile of at most 128 rows leaves group 1 without work, and the multiplying
// slots of group 0 then follow each other at once: it takes little over half the time.
#pragma once

#include "products.hpp"

namespace rs {

typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kWideThreads = 512;
constexpr int kWide = 256;              // results of a tile each way
constexpr int kStageBytes = 64;         // of c in a stage
constexpr int kWideOperand = kWide * kStageBytes;
constexpr int kRing = 4;
constexpr int kWideLds = kRing * 2 * kWideOperand;

typedef __attribute__((address_space(3))) void *lds_ptr;

__device__ __forceinline__ unsigned lds_address(const void *p) {
    return static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// Byte of a stage of an operand where 16-byte chunk `chunk` of its row `row`
// stands.  Along c a row is one of 256 and has 4 chunks; across it is one of 32
// steps of c and has 32 chunks, exchanged in fours of pairs, as the transposing read
// takes 32 bytes of a row.  The lanes that LDS serves at once (256 bytes: 16 of the
// wide reads, 32 of the transposing ones) meet every bank once: 246 bytes a clock and
// CU, 126 where two meet.
template <bool ACROSS>
__device__ __forceinline__ int stage_at(int row, int chunk) {
    if constexpr (!ACROSS) {
        return row * 64 + ((chunk ^ (row >> 2 & 3)) << 4);
    } else {
        return row * 512 + ((chunk ^ ((row & 3) << 2)) << 4);
    }
}

// Where a lane's reads of 32 rows or columns from mn on begin.  Along: at[k] for
// step k, rows 32 j further on are 2048 j bytes further.  Across: at[j] for the columns
// 32 j further on; 8192 bytes a step.
template <bool ACROSS>
struct Reader {
    unsigned at[ACROSS ? 4 : 2];

    __device__ __forceinline__ void set(int mn, int lane) {
        if constexpr (!ACROSS) {
            const int row = mn + (lane & 31), odd = lane >> 5;
            at[0] = stage_at<false>(row, odd);
            at[1] = stage_at<false>(row, 2 + odd);
        } else {
            const int i = lane & 15, g = lane >> 4;
            const int row = 8 * (g >> 1) + (i >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = mn + 32 * j + 16 * (g & 1);
                at[j] = stage_at<true>(row, (col >> 3) + (i >> 1 & 1)) + (i & 1) * 8;
            }
        }
    }
};

__device__ __forceinline__ i32x4 joined(i32x2 a, i32x2 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3); }

// The operands of a stage of a wave: p of 2 x 32 and q of 4 x 32 rows, 2 steps of 16
// elements of c.  The reads and the wait for them are one block, so that the compiler
// neither waits for the loads into LDS before it nor uses a register too early.
struct StageOperands {
    i32x4 p[2][2], q[4][2];
};

template <bool Q_ACROSS, bool P_ACROSS>
__device__ __forceinline__ void read_stage(const Reader<Q_ACROSS> &rq, const Reader<P_ACROSS> &rp, unsigned q_base,
                                           unsigned p_base, StageOperands &s) {
#if defined(__HIP_DEVICE_COMPILE__)  // (the host's pass knows no such registers)
    if constexpr (!Q_ACROSS && !P_ACROSS) {
        asm volatile(
            "ds_read_b128 %0, %12\n ds_read_b128 %4, %14\n ds_read_b128 %5, %14 offset:2048\n"
            "ds_read_b128 %6, %14 offset:4096\n ds_read_b128 %7, %14 offset:6144\n ds_read_b128 %1, %12 offset:2048\n"
            "ds_read_b128 %2, %13\n ds_read_b128 %3, %13 offset:2048\n ds_read_b128 %8, %15\n"
            "ds_read_b128 %9, %15 offset:2048\n ds_read_b128 %10, %15 offset:4096\n ds_read_b128 %11, %15 offset:6144\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(s.p[0][0]), "=&v"(s.p[1][0]), "=&v"(s.p[0][1]), "=&v"(s.p[1][1]), "=&v"(s.q[0][0]),
              "=&v"(s.q[1][0]), "=&v"(s.q[2][0]), "=&v"(s.q[3][0]), "=&v"(s.q[0][1]), "=&v"(s.q[1][1]),
              "=&v"(s.q[2][1]), "=&v"(s.q[3][1])
            : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(q_base + rq.at[0]), "v"(q_base + rq.at[1])
            : "memory");
    } else if constexpr (!Q_ACROSS) {
        i32x2 p[2][2][2];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16\n ds_read_b64_tr_b16 %1, %16 offset:2048\n"
            "ds_read_b128 %8, %18\n ds_read_b128 %9, %18 offset:2048\n ds_read_b128 %10, %18 offset:4096\n"
            "ds_read_b128 %11, %18 offset:6144\n"
            "ds_read_b64_tr_b16 %4, %17\n ds_read_b64_tr_b16 %5, %17 offset:2048\n"
            "ds_read_b64_tr_b16 %2, %16 offset:8192\n ds_read_b64_tr_b16 %3, %16 offset:10240\n"
            "ds_read_b64_tr_b16 %6, %17 offset:8192\n ds_read_b64_tr_b16 %7, %17 offset:10240\n"
            "ds_read_b128 %12, %19\n ds_read_b128 %13, %19 offset:2048\n ds_read_b128 %14, %19 offset:4096\n"
            "ds_read_b128 %15, %19 offset:6144\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(p[0][0][0]), "=&v"(p[0][0][1]), "=&v"(p[0][1][0]), "=&v"(p[0][1][1]), "=&v"(p[1][0][0]),
              "=&v"(p[1][0][1]), "=&v"(p[1][1][0]), "=&v"(p[1][1][1]), "=&v"(s.q[0][0]), "=&v"(s.q[1][0]),
              "=&v"(s.q[2][0]), "=&v"(s.q[3][0]), "=&v"(s.q[0][1]), "=&v"(s.q[1][1]), "=&v"(s.q[2][1]),
              "=&v"(s.q[3][1])
            : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(q_base + rq.at[0]), "v"(q_base + rq.at[1])
            : "memory");
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int k = 0; k < 2; ++k) s.p[j][k] = joined(p[j][k][0], p[j][k][1]);
        }
    } else {
        static_assert(Q_ACROSS && P_ACROSS);
        i32x2 p[2][2][2], q[4][2][2];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %24\n ds_read_b64_tr_b16 %1, %24 offset:2048\n"
            "ds_read_b64_tr_b16 %8, %26\n ds_read_b64_tr_b16 %9, %26 offset:2048\n"
            "ds_read_b64_tr_b16 %12, %27\n ds_read_b64_tr_b16 %13, %27 offset:2048\n"
            "ds_read_b64_tr_b16 %16, %28\n ds_read_b64_tr_b16 %17, %28 offset:2048\n"
            "ds_read_b64_tr_b16 %20, %29\n ds_read_b64_tr_b16 %21, %29 offset:2048\n"
            "ds_read_b64_tr_b16 %4, %25\n ds_read_b64_tr_b16 %5, %25 offset:2048\n"
            "ds_read_b64_tr_b16 %2, %24 offset:8192\n ds_read_b64_tr_b16 %3, %24 offset:10240\n"
            "ds_read_b64_tr_b16 %10, %26 offset:8192\n ds_read_b64_tr_b16 %11, %26 offset:10240\n"
            "ds_read_b64_tr_b16 %14, %27 offset:8192\n ds_read_b64_tr_b16 %15, %27 offset:10240\n"
            "ds_read_b64_tr_b16 %18, %28 offset:8192\n ds_read_b64_tr_b16 %19, %28 offset:10240\n"
            "ds_read_b64_tr_b16 %22, %29 offset:8192\n ds_read_b64_tr_b16 %23, %29 offset:10240\n"
            "ds_read_b64_tr_b16 %6, %25 offset:8192\n ds_read_b64_tr_b16 %7, %25 offset:10240\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(p[0][0][0]), "=&v"(p[0][0][1]), "=&v"(p[0][1][0]), "=&v"(p[0][1][1]), "=&v"(p[1][0][0]),
              "=&v"(p[1][0][1]), "=&v"(p[1][1][0]), "=&v"(p[1][1][1]), "=&v"(q[0][0][0]), "=&v"(q[0][0][1]),
              "=&v"(q[0][1][0]), "=&v"(q[0][1][1]), "=&v"(q[1][0][0]), "=&v"(q[1][0][1]), "=&v"(q[1][1][0]),
              "=&v"(q[1][1][1]), "=&v"(q[2][0][0]), "=&v"(q[2][0][1]), "=&v"(q[2][1][0]), "=&v"(q[2][1][1]),
              "=&v"(q[3][0][0]), "=&v"(q[3][0][1]), "=&v"(q[3][1][0]), "=&v"(q[3][1][1])
            : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(q_base + rq.at[0]), "v"(q_base + rq.at[1]),
              "v"(q_base + rq.at[2]), "v"(q_base + rq.at[3])
            : "memory");
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) s.p[j][k] = joined(p[j][k][0], p[j][k][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.q[j][k] = joined(q[j][k][0], q[j][k][1]);
        }
    }
#endif
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

// The same pointer in every lane, in scalar registers.
template <class T>
__device__ __forceinline__ const T *uniform(const T *p) {
    const auto bits = reinterpret_cast<uintptr_t>(p);
    const auto lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits)));
    const auto hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits >> 32)));
    return reinterpret_cast<const T *>(static_cast<uintptr_t>(hi) << 32 | lo);
}

// An operand on its way into LDS: a wave brings 2 x 1 KiB of a stage.
template <class T, bool ACROSS>
struct Feeder {
    static constexpr int kStep = kStageBytes / static_cast<int>(sizeof(T));
    unsigned offset[2];  // bytes from the tile's first element of a stage
    const T *base;       // of the next stage
    size_t stride;
    int rows, width, row0, col0;

    // Row and column in the tile of the 16 bytes that a lane brings in load i.
    // Rows and columns of results that do not exist are others' again.
    __device__ __forceinline__ void place(int i, int wave, int lane, int &row, int &col) const {
        if constexpr (!ACROSS) {
            const int r = (2 * wave + i) * 16 + (lane >> 2);
            row = r < rows - row0 ? r : rows - row0 - 1;
            col = ((lane & 3) ^ (r >> 2 & 3)) * 8;
        } else {
            row = (2 * wave + i) * 2 + (lane >> 5);
            const int c = ((lane & 31) ^ ((row & 3) << 2)) * 8;
            col = c < width - col0 - 8 ? c : width - col0 - 8;
        }
    }

    // The operand's matrix has `rows` rows of `width` elements, the tile begins at
    // `first`, a row (along) or a column (across).
    __device__ __forceinline__ void set(const T *matrix, size_t stride_, int rows_, int width_, int first, int wave,
                                        int lane) {
        stride = stride_, rows = rows_, width = width_;
        row0 = ACROSS ? 0 : first, col0 = ACROSS ? first : 0;
        base = uniform(matrix + static_cast<size_t>(row0) * stride + col0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int row, col;
            place(i, wave, lane, row, col);
            offset[i] = static_cast<unsigned>((static_cast<size_t>(row) * stride + col) * sizeof(T));
        }
    }

    // Enqueues the loads of the next stage to `to`.
    __device__ __forceinline__ void load(char *to, int wave) {
        const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(base), 0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)(to + (2 * wave + i) * 1024), 16,
                                                     static_cast<int>(offset[i]), 0, 0, 0);
        }
        base += ACROSS ? kStep * stride : kStep;
    }

    // The last stage, of which `have` elements of c exist: through registers, zeros
    // behind them.
    __device__ __forceinline__ void load_part(char *to, int wave, int lane, int have) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int row, col;
            place(i, wave, lane, row, col);
            i32x4 v;
            if constexpr (!ACROSS) {
                // From the row's last whole chunk at most (the row has one).
                const int back = have - 8 < col ? have - 8 : col;
                v = load16(reinterpret_cast<const char *>(base + static_cast<size_t>(row) * stride + back));
                v = cut<T>(v, col, have);
            } else {
                const int r = row < have ? row : 0;
                v = load16(reinterpret_cast<const char *>(base + static_cast<size_t>(r) * stride + col));
                if (row >= have) v = i32x4{0, 0, 0, 0};
            }
            *reinterpret_cast<i32x4 *>(to + (2 * wave + i) * 1024 + lane * 16) = v;
        }
    }
};

// ---------------------------------------------------------------------------
// Which tile a workgroup takes.  Consecutive workgroups go to the eight XCDs in
// turn, each with an L2 of its own: XCD x takes tiles that stand together.  Within an
// expert they go over kTurn tiles of q, then p, so that the 32 workgroups of an XCD share
// both operands.
// ---------------------------------------------------------------------------
constexpr int kXcds = 8;
constexpr int kTurn = 4;

struct WideTile {
    int expert;  // -1: none; `experts`: rows of no expert
    int q, p;    // tiles
    RowSpan rows;
};

__device__ __forceinline__ void within(int local, int q_tiles, int p_tiles, WideTile &t) {
    const int turn = local / (kTurn * p_tiles), left = q_tiles - turn * kTurn, r = local - turn * kTurn * p_tiles;
    const int deep = left < kTurn ? left : kTurn;
    t.q = turn * kTurn + r % deep;
    t.p = r / deep;
}

// Of ragged rows: block b of `grid` workgroups.
__device__ inline WideTile wide_rows_tile(const int32_t *offsets, int experts, int num_rows, int height, int p_tiles,
                                          bool clear, unsigned b) {
    WideTile t{-1, 0, 0, {0, num_rows}};
    const int lane = threadIdx.x & 63;
    int all = 0, before = 0, from = num_rows;
    if (offsets == nullptr) {
        all = tiles_of(num_rows, height);
    } else {
        for (int base = 0; base < experts; base += 64) {
            const RowSpan r = rows_of(offsets, base + lane < experts ? base + lane : experts - 1, num_rows);
            const int tiles = base + lane < experts ? tiles_of(r.hi - r.lo, height) : 0;
            all += __builtin_amdgcn_readlane(wave_prefix(tiles, lane), 63);
        }
        before = row_bound(offsets, 0, num_rows), from = row_bound(offsets, experts, num_rows);
        from = from < before ? before : from;
    }
    const int rest = clear ? tiles_of(before + (num_rows - from), height) : 0;
    const unsigned jobs = static_cast<unsigned>(all + rest) * static_cast<unsigned>(p_tiles);
    const unsigned chunk = (jobs + kXcds - 1) / kXcds, at = b / kXcds;
    unsigned job = b % kXcds * chunk + at;
    if (at >= chunk || job >= jobs) return t;
    if (offsets == nullptr) {
        t.expert = 0;
        within(static_cast<int>(job), all, p_tiles, t);
        return t;
    }
    if (job >= static_cast<unsigned>(all) * p_tiles) {
        t.expert = experts;
        t.rows = {before, from};
        within(static_cast<int>(job - static_cast<unsigned>(all) * p_tiles), rest, p_tiles, t);
        return t;
    }
    int tile = static_cast<int>(job / p_tiles);
    for (int base = 0; base < experts; base += 64) {
        const RowSpan r = rows_of(offsets, base + lane < experts ? base + lane : experts - 1, num_rows);
        const int tiles = base + lane < experts ? tiles_of(r.hi - r.lo, height) : 0;
        const int upto = wave_prefix(tiles, lane), sum = __builtin_amdgcn_readlane(upto, 63);
        if (tile < sum) {
            const int found = __ffsll(static_cast<unsigned long long>(__ballot(upto > tile))) - 1;
            const int first = __builtin_amdgcn_readlane(upto - tiles, found);
            t.expert = base + found;
            t.rows = {__builtin_amdgcn_readlane(r.lo, found), __builtin_amdgcn_readlane(r.hi, found)};
            // (Tiles before this chunk of experts are gone from `tile`, not from `job`.)
            const unsigned gone = job / p_tiles - static_cast<unsigned>(tile);
            within(static_cast<int>(job - (gone + first) * static_cast<unsigned>(p_tiles)),
                   __builtin_amdgcn_readlane(tiles, found), p_tiles, t);
            return t;
        }
        tile -= sum;
    }
    return t;
}

// Of the weights' gradient: every expert has the same tiles.
__device__ inline WideTile wide_weights_tile(int experts, int q_tiles, int p_tiles, unsigned b) {
    WideTile t{-1, 0, 0, {0, 0}};
    const unsigned tiles = static_cast<unsigned>(q_tiles) * static_cast<unsigned>(p_tiles);
    const unsigned chunk = (tiles + kXcds - 1) / kXcds, e = b / (chunk * kXcds), local = b % (chunk * kXcds);
    const unsigned job = local % kXcds * chunk + local / kXcds;
    if (e >= static_cast<unsigned>(experts) || job >= tiles) return t;
    t.expert = static_cast<int>(e);
    within(static_cast<int>(job), q_tiles, p_tiles, t);
    return t;
}

template <class T, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS>
__global__ __launch_bounds__(kWideThreads) void wide_product_kernel(const ProductWork<T, T> w) {
    __shared__ __align__(1024) char ring[kWideLds];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = wave >> 2, q_wave = group * 128, p_wave = (wave & 3) * 64;
    const int num_rows = static_cast<int>(w.num_rows), p_tiles = (w.pn + kWide - 1) / kWide;

    const T *q = w.q, *p = w.p;
    T *out = w.out;
    int q_rows, c_n;
    const WideTile t = RAGGED_C
        ? wide_weights_tile(w.experts, (w.qn + kWide - 1) / kWide, p_tiles, blockIdx.x)
        : wide_rows_tile(w.offsets, w.experts, num_rows, kWide, p_tiles, w.clear, blockIdx.x);
    if (t.expert < 0) return;
    const int q0 = t.q * kWide, p0 = t.p * kWide;
    if constexpr (RAGGED_C) {
        const RowSpan r = rows_of(w.offsets, t.expert, num_rows);
        q_rows = w.qn;
        c_n = r.hi - r.lo;
        q += static_cast<size_t>(r.lo) * w.q_stride;
        p += static_cast<size_t>(r.lo) * w.p_stride;
        out += static_cast<size_t>(t.expert) * w.out_expert;
    } else {
        if (t.expert == w.experts) {
            clear_tile(out, w.out_stride, w.pn, RowTile{t.expert, t.q, t.rows}, kWide, num_rows, p0, kWide);
            return;
        }
        q_rows = t.rows.hi - t.rows.lo;
        c_n = w.cn;
        q += static_cast<size_t>(t.rows.lo) * w.q_stride;
        out += static_cast<size_t>(t.rows.lo) * w.out_stride;
        p += static_cast<size_t>(t.expert) * w.p_expert;
    }

    if (q0 >= q_rows || p0 >= w.pn) return;

    constexpr int kStep = kStageBytes / static_cast<int>(sizeof(T));
    const int stages = (c_n + kStep - 1) / kStep;
    f32x16 acc[2][4];
#pragma unroll
    for (auto &a : acc) {
#pragma unroll
        for (auto &b : a) {
#pragma unroll
            for (int i = 0; i < 16; ++i) b[i] = 0.0f;
        }
    }
    if (stages > 0) {
        Feeder<T, Q_ACROSS> fq;
        Feeder<T, P_ACROSS> fp;
        fq.set(q, w.q_stride, Q_ACROSS ? c_n : q_rows, Q_ACROSS ? w.qn : c_n, q0, wave, lane);
        fp.set(p, w.p_stride, P_ACROSS ? c_n : w.pn, P_ACROSS ? w.pn : c_n, p0, wave, lane);
        Reader<Q_ACROSS> rq;
        Reader<P_ACROSS> rp;
        rq.set(q_wave, lane);
        rp.set(p_wave, lane);
        const unsigned lds = lds_address(ring);
        // Whether this wave has results at all.
        const bool works = q0 + q_wave < q_rows && p0 + p_wave < w.pn;

        const auto issue = [&](int s) {
            char *to = ring + s % kRing * (2 * kWideOperand);
            const int have = c_n - s * kStep;
            if (have >= kStep) {
                fq.load(to, wave);
                fp.load(to + kWideOperand, wave);
            } else {
                fq.load_part(to, wave, lane, have);
                fp.load_part(to + kWideOperand, wave, lane, have);
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            }
        };
        // Waits until of the stages enqueued last only `late` are on their way: four
        // loads each.
        const auto wait = [&](int late) {
            if (late >= 2) {
                asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
            } else if (late == 1) {
                asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
        };
        const auto barrier = [] {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        const int first = stages < 3 ? stages : 3;
        for (int s = 0; s < first; ++s) issue(s);
        wait(first - 1);
        barrier();
        if (group == 1) barrier();  // half a turn behind
        for (int s = 0; s < stages; ++s) {
            // The place of stage s + 3 was read last, by group 1, in the slot before this one.
            if (s + 3 < stages) issue(s + 3);
            StageOperands o;
            const unsigned at = lds + static_cast<unsigned>(s % kRing) * (2 * kWideOperand);
            if (works) read_stage<Q_ACROSS, P_ACROSS>(rq, rp, at, at + kWideOperand, o);
            wait(stages - 2 - s);
            barrier();
            if (works) {
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = mma32<T>(o.p[i][k], o.q[j][k], acc[i][j]);
                    }
                }
                __builtin_amdgcn_s_setprio(0);
            }
            barrier();
        }
        if (group == 0) barrier();
    }

    // Results to rows: through the wave's 16 KiB of the ring, 128 rows of 64
    // elements, so that 8 lanes write 128 bytes of a row.
    __syncthreads();
    char *mine = ring + wave * 16384;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 32 * j + (lane & 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                typedef T t4 __attribute__((ext_vector_type(4)));
                t4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = static_cast<T>(acc[i][j][4 * a + r]);
                const int chunk = 4 * i + a;
                *reinterpret_cast<t4 *>(mine + row * 128 + ((chunk ^ (row & 7)) << 4) + (lane >> 5) * 8) = v;
            }
        }
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
        const int row = 8 * k + (lane >> 3), chunk = lane & 7;
        const i32x4 v = *reinterpret_cast<const i32x4 *>(mine + row * 128 + ((chunk ^ (row & 7)) << 4));
        const int qi = q0 + q_wave + row, pi = p0 + p_wave + 8 * chunk, have = w.pn - pi;
        if (qi >= q_rows || have <= 0) continue;
        T *to = out + static_cast<size_t>(qi) * w.out_stride + pi;
        if (have >= 8) {
            *reinterpret_cast<i32x4_any *>(to) = v;
        } else {
            union {
                i32x4 all;
                T e[8];
            } u{v};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e < have) to[e] = u.e[e];
            }
        }
    }
}

}  // namespace rs
