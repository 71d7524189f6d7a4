// products_wide.hpp -- the experts' products in 16 bits for many rows an expert:
// 256 x 256 results a workgroup of eight waves, operands brought to LDS by the
// memory system itself, without passing through registers.
//
// The waves form two groups of four, one wave of each group on every SIMD.  Each group
// has half of the rows q, each of its waves 64 columns p, so a wave holds 128 x 64
// results.  The contraction goes in stages of 128 bytes of c (whole
// cache lines), two slots each: the first 64 rows of a group, then the other 64.  In a
// slot, one group reads what it needs from LDS while the other multiplies; a barrier
// ends the slot and they change places, so a SIMD multiplies in every slot.
// LDS holds two stages.  What a slot has read, p and the first rows or the
// others, is loaded again at once, and has five slots to arrive.
//
// A tile with fewer rows is shared evenly, in 32s: its time goes with its rows in steps
// of 64.  One of at most 128 has no second rows: a stage is then one slot, and three
// fit into LDS.
#pragma once

#include "products.hpp"

namespace rs {

typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kWideThreads = 512;
constexpr int kWide = 256;              // results of a tile each way
constexpr int kStageBytes = 128;        // of c in a stage
constexpr int kWideOperand = kWide * kStageBytes;
constexpr int kWideStage = 2 * kWideOperand;  // p, the first 64 rows q of both groups, their others
constexpr int kFlatStage = kWideStage * 3 / 4;  // without the others
constexpr int kWideLds = 3 * kFlatStage;      // three of the latter, two of the former

typedef __attribute__((address_space(3))) void *lds_ptr;

__device__ __forceinline__ unsigned lds_address(const void *p) {
    return static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// Byte of a block of LDS where 16-byte chunk `chunk` of its row `row` stands.  Along
// c a row has 8 chunks; across it is a step of c with 32 chunks (p) or 16 (half of
// q), exchanged in fours, as the transposing read takes 32 bytes of a row.  The lanes that
// LDS serves at once (256 bytes: 16 of the wide reads, 32 of the transposing ones)
// meet every bank once: 246 bytes a clock and CU, 126 where two meet.
template <bool ACROSS, int CHUNKS>
__device__ __forceinline__ int stage_at(int row, int chunk) {
    static_assert(ACROSS || CHUNKS == 8);
    const int turn = ACROSS ? (row & 3) << 2 : row >> 1 & 7;
    return row * (CHUNKS * 16) + ((chunk ^ turn) << 4);
}

// Where a lane's reads of 2 x 32 rows or columns from mn on begin.  Along: at[k] for
// step k of 16 elements of c, and 4096 bytes further for the second 32 rows.
// Across: at[j] for the j-th 32 columns, a step is 16 rows further.
template <bool ACROSS, int CHUNKS>
struct Reader {
    unsigned at[ACROSS ? 2 : 4];

    __device__ __forceinline__ void set(int mn, int lane) {
        if constexpr (!ACROSS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) at[k] = stage_at<false, CHUNKS>(mn + (lane & 31), 2 * k + (lane >> 5));
        } else {
            const int i = lane & 15, g = lane >> 4;
            const int row = 8 * (g >> 1) + (i >> 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = mn + 32 * j + 16 * (g & 1);
                at[j] = stage_at<true, CHUNKS>(row, (col >> 3) + (i >> 1 & 1)) + (i & 1) * 8;
            }
        }
    }
};

__device__ __forceinline__ i32x4 joined(i32x2 a, i32x2 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3); }

// Operands of 2 x 32 rows, 4 steps of 16 elements of c.
struct Operands {
    i32x4 f[2][4];
};

// Reads of an operand's block and the wait for them, one block of instructions, so
// that the compiler neither waits for the loads into LDS before it nor uses a register
// too early.
#if defined(__HIP_DEVICE_COMPILE__)  // (the host's pass knows no such registers)
#define RS_READ_ALONG(n0, n1, n2, n3, n4, n5, n6, n7, a0, a1, a2, a3)                                    \
    "ds_read_b128 %" #n0 ", %" #a0 "\n ds_read_b128 %" #n4 ", %" #a0 " offset:4096\n"                    \
    "ds_read_b128 %" #n1 ", %" #a1 "\n ds_read_b128 %" #n5 ", %" #a1 " offset:4096\n"                    \
    "ds_read_b128 %" #n2 ", %" #a2 "\n ds_read_b128 %" #n6 ", %" #a2 " offset:4096\n"                    \
    "ds_read_b128 %" #n3 ", %" #a3 "\n ds_read_b128 %" #n7 ", %" #a3 " offset:4096\n"
#define RS_ALONG_OUT(o)                                                                                   \
    "=&v"(o.f[0][0]), "=&v"(o.f[0][1]), "=&v"(o.f[0][2]), "=&v"(o.f[0][3]), "=&v"(o.f[1][0]), "=&v"(o.f[1][1]), \
        "=&v"(o.f[1][2]), "=&v"(o.f[1][3])
#define RS_READ_TURNED(n, a, o) "ds_read_b64_tr_b16 %" #n ", %" #a " offset:" #o "\n"
#define RS_TURNED_OUT(v)                                                                                  \
    "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]), \
        "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11]), "=&v"(v[12]), "=&v"(v[13]), "=&v"(v[14]), "=&v"(v[15])
#endif

__device__ __forceinline__ void from_turned(const i32x2 (&v)[16], Operands &o) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o.f[j][k] = joined(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
    }
}

// q alone.
template <bool Q_ACROSS>
__device__ __forceinline__ void read_q(const Reader<Q_ACROSS, Q_ACROSS ? 16 : 8> &r, unsigned base, Operands &o) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (!Q_ACROSS) {
        asm volatile(RS_READ_ALONG(0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11) "s_waitcnt lgkmcnt(0)"
                     : RS_ALONG_OUT(o)
                     : "v"(base + r.at[0]), "v"(base + r.at[1]), "v"(base + r.at[2]), "v"(base + r.at[3])
                     : "memory");
    } else {
        i32x2 v[16];
        asm volatile(RS_READ_TURNED(0, 16, 0) RS_READ_TURNED(1, 16, 1024) RS_READ_TURNED(8, 17, 0)
                     RS_READ_TURNED(9, 17, 1024) RS_READ_TURNED(2, 16, 4096) RS_READ_TURNED(3, 16, 5120)
                     RS_READ_TURNED(10, 17, 4096) RS_READ_TURNED(11, 17, 5120) RS_READ_TURNED(4, 16, 8192)
                     RS_READ_TURNED(5, 16, 9216) RS_READ_TURNED(12, 17, 8192) RS_READ_TURNED(13, 17, 9216)
                     RS_READ_TURNED(6, 16, 12288) RS_READ_TURNED(7, 16, 13312) RS_READ_TURNED(14, 17, 12288)
                     RS_READ_TURNED(15, 17, 13312) "s_waitcnt lgkmcnt(0)"
                     : RS_TURNED_OUT(v)
                     : "v"(base + r.at[0]), "v"(base + r.at[1])
                     : "memory");
        from_turned(v, o);
    }
#endif
}

// p and q.
template <bool Q_ACROSS, bool P_ACROSS>
__device__ __forceinline__ void read_pq(const Reader<Q_ACROSS, Q_ACROSS ? 16 : 8> &rq,
                                        const Reader<P_ACROSS, P_ACROSS ? 32 : 8> &rp, unsigned q_base,
                                        unsigned p_base, Operands &q, Operands &p) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (!P_ACROSS) {
        static_assert(!Q_ACROSS);
        asm volatile(RS_READ_ALONG(0, 1, 2, 3, 4, 5, 6, 7, 16, 17, 18, 19)
                     RS_READ_ALONG(8, 9, 10, 11, 12, 13, 14, 15, 20, 21, 22, 23) "s_waitcnt lgkmcnt(0)"
                     : RS_ALONG_OUT(p), RS_ALONG_OUT(q)
                     : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(p_base + rp.at[2]), "v"(p_base + rp.at[3]),
                       "v"(q_base + rq.at[0]), "v"(q_base + rq.at[1]), "v"(q_base + rq.at[2]), "v"(q_base + rq.at[3])
                     : "memory");
    } else {
#define RS_READ_TURNED_P(a, b)                                                                                     \
    RS_READ_TURNED(0, a, 0) RS_READ_TURNED(1, a, 2048) RS_READ_TURNED(8, b, 0) RS_READ_TURNED(9, b, 2048)             \
    RS_READ_TURNED(2, a, 8192) RS_READ_TURNED(3, a, 10240) RS_READ_TURNED(10, b, 8192)                              \
    RS_READ_TURNED(11, b, 10240) RS_READ_TURNED(4, a, 16384) RS_READ_TURNED(5, a, 18432)                            \
    RS_READ_TURNED(12, b, 16384) RS_READ_TURNED(13, b, 18432) RS_READ_TURNED(6, a, 24576)                           \
    RS_READ_TURNED(7, a, 26624) RS_READ_TURNED(14, b, 24576) RS_READ_TURNED(15, b, 26624)
        i32x2 v[16];
        if constexpr (!Q_ACROSS) {
            asm volatile(RS_READ_TURNED_P(24, 25) RS_READ_ALONG(16, 17, 18, 19, 20, 21, 22, 23, 26, 27, 28, 29)
                         "s_waitcnt lgkmcnt(0)"
                         : RS_TURNED_OUT(v), RS_ALONG_OUT(q)
                         : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(q_base + rq.at[0]),
                           "v"(q_base + rq.at[1]), "v"(q_base + rq.at[2]), "v"(q_base + rq.at[3])
                         : "memory");
        } else {
            asm volatile(RS_READ_TURNED_P(16, 17) "s_waitcnt lgkmcnt(0)"
                         : RS_TURNED_OUT(v)
                         : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1])
                         : "memory");
            read_q<true>(rq, q_base, q);
        }
        from_turned(v, p);
    }
#endif
}

// The same pointer in every lane, in scalar registers.
template <class T>
__device__ __forceinline__ const T *uniform(const T *p) {
    const auto bits = reinterpret_cast<uintptr_t>(p);
    const auto lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits)));
    const auto hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bits >> 32)));
    return reinterpret_cast<const T *>(static_cast<uintptr_t>(hi) << 32 | lo);
}

// A block of an operand on its way into LDS, a KiB a wave and load: p, 4 loads, or half
// (0, 1) of q, 2 loads: 64 rows of each group.
template <class T, bool ACROSS, bool IS_P>
struct Feeder {
    static constexpr int kLoads = IS_P ? 4 : 2;
    static constexpr int kChunks = ACROSS ? (IS_P ? 32 : 16) : 8;
    static constexpr int kRows = 64 / kChunks;  // of LDS in a load
    static constexpr int kStep = kStageBytes / static_cast<int>(sizeof(T));
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    unsigned offset[kLoads];  // bytes from the tile's first element of a stage
    const T *base;            // of the next stage
    size_t stride;
    int rows, width, first, half, height;

    // Row or column of the tile that row or column i of the block is.
    __device__ __forceinline__ int of_tile(int i) const { return IS_P ? i : (i >> 6) * height + half * 64 + (i & 63); }

    // Row and column in the tile of the 16 bytes that a lane brings in load i.
    // Rows and columns of results that do not exist are others' again.
    __device__ __forceinline__ void place(int i, int wave, int lane, int &row, int &col) const {
        const int r = (kLoads * wave + i) * kRows + lane / kChunks, c = lane % kChunks;
        if constexpr (!ACROSS) {
            const int t = of_tile(r), last = rows - first - 1;
            row = t < last ? t : last;
            col = (c ^ (r >> 1 & 7)) * V;
        } else {
            const int t = of_tile((c ^ ((r & 3) << 2)) * V), last = width - first - V;
            row = r;
            col = t < last ? t : last;
        }
    }

    // The operand's matrix has `rows` rows of `width` elements, the tile begins at
    // `first`, a row (along) or a column (across), and a group has `height` rows q.
    __device__ __forceinline__ void set(const T *matrix, size_t stride_, int rows_, int width_, int first_, int half_,
                                        int height_, int wave, int lane) {
        stride = stride_, rows = rows_, width = width_, first = first_, half = half_, height = height_;
        base = uniform(matrix + (ACROSS ? static_cast<size_t>(first) : static_cast<size_t>(first) * stride));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int row, col;
            place(i, wave, lane, row, col);
            offset[i] = static_cast<unsigned>((static_cast<size_t>(row) * stride + col) * sizeof(T));
        }
    }

    // Enqueues the loads of the next stage, of which `have` elements of c exist, to
    // `to`.  The last ones go through registers, with zeros behind them.
    __device__ __forceinline__ void load(char *to, int wave, int lane, int have) {
        if (have >= kStep) {
            const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(base), 0, 0x7FFFFFFF, 0x00020000);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)(to + (kLoads * wave + i) * 1024), 16,
                                                         static_cast<int>(offset[i]), 0, 0, 0);
            }
            base += ACROSS ? kStep * stride : kStep;
            return;
        }
        int own = lane;
#if defined(__HIP_DEVICE_COMPILE__)
        asm volatile("" : "+v"(own));  // keeps what follows from being worked out, and held, before the loop
#endif
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int row, col;
            place(i, wave, own, row, col);
            i32x4 v;
            if constexpr (!ACROSS) {
                // From the row's last whole chunk at most (the row has one).
                const int back = have - V < col ? have - V : col;
                v = load16(reinterpret_cast<const char *>(base + static_cast<size_t>(row) * stride + back));
                v = cut<T>(v, col, have);
            } else {
                const int r = row < have ? row : 0;
                v = load16(reinterpret_cast<const char *>(base + static_cast<size_t>(r) * stride + col));
                if (row >= have) v = i32x4{0, 0, 0, 0};
            }
            *reinterpret_cast<i32x4 *>(to + (kLoads * wave + i) * 1024 + lane * 16) = v;
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
};

template <class T, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS>
__global__ __launch_bounds__(kWideThreads) void wide_product_kernel(const ProductWork<T, T> w) {
    __shared__ __align__(1024) char ring[kWideLds];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = wave >> 2, p_wave = (wave & 3) * 64;
    const int num_rows = static_cast<int>(w.num_rows), p_tiles = (w.pn + kWide - 1) / kWide;

    const T *q = w.q, *p = w.p;
    T *out = w.out;
    int q_rows, c_n;
    const ResultTile t = RAGGED_C
        ? weights_tile(w.experts, (w.qn + kWide - 1) / kWide, p_tiles, blockIdx.x)
        : rows_tile(w.offsets, w.experts, num_rows, kWide, p_tiles, w.clear, blockIdx.x);
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
    // Rows of a group: half of the tile's, in 32s.
    const int left = q_rows - q0 < kWide ? q_rows - q0 : kWide;
    const int height = (left + 63) / 64 * 32, q_wave = group * height;

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
        Feeder<T, Q_ACROSS, false> f0, f1;
        Feeder<T, P_ACROSS, true> fp;
        f0.set(q, w.q_stride, Q_ACROSS ? c_n : q_rows, Q_ACROSS ? w.qn : c_n, q0, 0, height, wave, lane);
        f1.set(q, w.q_stride, Q_ACROSS ? c_n : q_rows, Q_ACROSS ? w.qn : c_n, q0, 1, height, wave, lane);
        fp.set(p, w.p_stride, P_ACROSS ? c_n : w.pn, P_ACROSS ? w.pn : c_n, p0, 0, 0, wave, lane);
        Reader<Q_ACROSS, Q_ACROSS ? 16 : 8> rq;
        Reader<P_ACROSS, P_ACROSS ? 32 : 8> rp;
        rq.set(group * 64, lane);
        rp.set(p_wave, lane);
        const unsigned lds = lds_address(ring);
        // Whether this wave has results at all.
        const bool works = q0 + q_wave < q_rows && p0 + p_wave < w.pn;

        // Six loads a wave: p and the first rows of stage s, to `to`; two: the others.
        const auto load0 = [&](int s, char *to) __attribute__((always_inline)) {
            fp.load(to, wave, lane, c_n - s * kStep);
            f0.load(to + kWideOperand, wave, lane, c_n - s * kStep);
        };
        const auto issue0 = [&](int s) __attribute__((always_inline)) {
            if (s < stages) load0(s, ring + s % 2 * kWideStage);
        };
        const auto issue1 = [&](int s) __attribute__((always_inline)) {
            if (s < stages) f1.load(ring + s % 2 * kWideStage + kWideOperand * 3 / 2, wave, lane, c_n - s * kStep);
        };
        // Waits for the first part of stage s (behind it its second and the first of the
        // next may be on their way), or for its second (behind it the whole next one).
        const auto arrived0 = [&](int s) __attribute__((always_inline)) {
            if (s + 1 < stages) {
                asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
            } else if (s < stages) {
                asm volatile("s_waitcnt vmcnt(2)" ::: "memory");
            }
        };
        const auto arrived1 = [&](int s) __attribute__((always_inline)) {
            if (s + 1 < stages) {
                asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
        };
        const auto barrier = []() __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        Operands op, oq;
        // Multiplies rows 64 HALF .. of the group, 32 times BLOCKS, with the operands read
        // last.
        const auto multiply = [&](int s, auto half, auto blocks) __attribute__((always_inline)) {
            constexpr int kHalf = decltype(half)::value, kBlocks = decltype(blocks)::value;
            const auto step = [&](int k) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        acc[i][2 * kHalf + j] = mma32<T>(op.f[i][k], oq.f[j][k], acc[i][2 * kHalf + j]);
                    }
                }
            };
            __builtin_amdgcn_s_setprio(1);
            step(0), step(1);
            if (c_n - s * kStep > kStep / 2) step(2), step(3);  // (zeros otherwise)
            __builtin_amdgcn_s_setprio(0);
        };
        constexpr std::integral_constant<int, 0> k0{};
        constexpr std::integral_constant<int, 1> k1{};
        constexpr std::integral_constant<int, 2> k2{};
        // Slots: group 0 reads in the even ones and multiplies in the odd ones, group 1
        // the other way round, a slot later.  Group 1 is the last to multiply, and nobody
        // waits for that.
        // Tiles of more than 128 rows.  What group 0 reads of stage s in slots 4 s and
        // 4 s + 2, group 1 has read at the end of slots 4 s + 1 and 4 s + 3: from then on
        // stage s + 2 takes its place.  Both groups have waited for it before group 0's slots
        // 4 s + 8 and 4 s + 10.
        const auto tall = [&](auto others) __attribute__((always_inline)) {
            issue0(0);
            issue1(0);
            issue0(1);
            if (stages > 1) {
                asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            barrier();
            if (group == 1) barrier();
#pragma nounroll
            for (int s = 0; s < stages; ++s) {
                const unsigned at = lds + static_cast<unsigned>(s % 2) * kWideStage;
                if (works) read_pq<Q_ACROSS, P_ACROSS>(rq, rp, at + kWideOperand, at, oq, op);
                issue1(s + 1);
                if (group == 1) arrived1(s);
                barrier();
                if (works) multiply(s, k0, k2);
                if (group == 0) arrived1(s);
                barrier();
                if (works) read_q<Q_ACROSS>(rq, at + kWideOperand * 3 / 2, oq);
                issue0(s + 2);
                if (group == 1) arrived0(s + 1);
                barrier();
                if (works) multiply(s, k1, others);
                if (group == 0) arrived0(s + 1);
                if (s + 1 < stages || group == 0) barrier();
            }
        };
        // The others.  Group 0 reads stage s in slot 2 s, group 1 in the next; from slot
        // 2 s + 2 on stage s + 3 takes its place.  It is read first in slot 2 s + 6.
        const auto flat = [&](auto rows) __attribute__((always_inline)) {
            const auto issue = [&](int s, unsigned place) __attribute__((always_inline)) {
                if (s < stages) load0(s, ring + place * kFlatStage);
            };
            const auto arrived = [&](int s) __attribute__((always_inline)) {  // behind stage s the next may be on its way
                if (s + 1 < stages) {
                    asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
                } else {
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                }
            };
            issue(0, 0);
            issue(1, 1);
            arrived(0);
            if (group == 1) issue(2, 2);
            barrier();
            if (group == 1) barrier();
            unsigned place = 0;
#pragma nounroll
            for (int s = 0; s < stages; ++s) {
                const unsigned at = lds + place * kFlatStage, before = place == 0 ? 2 : place - 1;
                if (works) read_pq<Q_ACROSS, P_ACROSS>(rq, rp, at + kWideOperand, at, oq, op);
                if (group == 0) {
                    issue(s + 2, before);
                } else {
                    arrived(s + 1);
                }
                barrier();
                if (group == 1) issue(s + 3, place);
                if (works) multiply(s, k0, rows);
                if (group == 0) arrived(s + 1);
                if (s + 1 < stages || group == 0) barrier();
                place = place == 2 ? 0 : place + 1;
            }
        };
        if (height == 128) {
            tall(k2);
        } else if (height == 96) {
            tall(k1);
        } else if (height == 64) {
            flat(k2);
        } else {
            flat(k1);
        }
    }

    // Results to rows: through the wave's own 16 KiB of LDS, 128 rows of 64
    // elements, so that 8 lanes write 128 bytes of a row.  (All operands have been
    // read: group 0 passed the barrier behind the slot in which group 1 read the last.)
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
                *reinterpret_cast<t4 *>(mine + result_at(row, chunk) + (lane >> 5) * 8) = v;
            }
        }
    }
    wave_exchange();
    rows_from_lds(mine, out, w.out_stride, height, q0 + q_wave, q_rows, p0 + p_wave, w.pn, lane);
}

// ---------------------------------------------------------------------------
// The same of operands in 8 bits: a stage is a block of 128 elements that share a
// scale.  Results of a block stand for themselves times the scales of row and
// matrix, and are added to the sums in float32: 16 x 16 of them at a time, while the next
// are multiplied.  The scales of the rows come with the stage.
// Results in bfloat16: the others' sums, taken whole, would need 320 conversions a slot here, as
// there are no registers for p in float16 (32768 rows of 32 x 4096 x 7168 3570 us, 2130 with square tiles).
// ---------------------------------------------------------------------------
// Scales of a stage: of the first 64 rows of both groups, then of their others, each
// with room for what the six waves bring whose loads nobody reads (all waves load as
// often, as they count their own).
constexpr int kScaleBytes = 4096;

struct Reader8 {
    unsigned at[2];

    __device__ __forceinline__ void set(int mn, int lane) {
#pragma unroll
        for (int k = 0; k < 2; ++k) at[k] = stage_at<false, 8>(mn + (lane & 15), 4 * k + (lane >> 4));
    }
};

// Operands of 4 x 16 rows, 128 elements of c, and the scales of rows q.
struct Operands8 {
    i32x4 f[4][2];
};

#if defined(__HIP_DEVICE_COMPILE__)
#define RS_READ_8(n0, n1, n2, n3, n4, n5, n6, n7, a0, a1)                                       \
    "ds_read_b128 %" #n0 ", %" #a0 "\n ds_read_b128 %" #n1 ", %" #a1 "\n"                       \
    "ds_read_b128 %" #n2 ", %" #a0 " offset:2048\n ds_read_b128 %" #n3 ", %" #a1 " offset:2048\n" \
    "ds_read_b128 %" #n4 ", %" #a0 " offset:4096\n ds_read_b128 %" #n5 ", %" #a1 " offset:4096\n" \
    "ds_read_b128 %" #n6 ", %" #a0 " offset:6144\n ds_read_b128 %" #n7 ", %" #a1 " offset:6144\n"
#define RS_READ_SCALES(n0, n1, n2, n3, a)                                        \
    "ds_read_b32 %" #n0 ", %" #a "\n ds_read_b32 %" #n1 ", %" #a " offset:64\n" \
    "ds_read_b32 %" #n2 ", %" #a " offset:128\n ds_read_b32 %" #n3 ", %" #a " offset:192\n"
#define RS_8_OUT(o)                                                                                               \
    "=&v"(o.f[0][0]), "=&v"(o.f[0][1]), "=&v"(o.f[1][0]), "=&v"(o.f[1][1]), "=&v"(o.f[2][0]), "=&v"(o.f[2][1]), \
        "=&v"(o.f[3][0]), "=&v"(o.f[3][1])
#endif

__device__ __forceinline__ void read_pq8(const Reader8 &rq, const Reader8 &rp, unsigned q_base, unsigned p_base,
                                         unsigned scales, Operands8 &q, Operands8 &p, float (&scale)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile(RS_READ_8(0, 1, 2, 3, 4, 5, 6, 7, 20, 21) RS_READ_8(8, 9, 10, 11, 12, 13, 14, 15, 22, 23)
                 RS_READ_SCALES(16, 17, 18, 19, 24) "s_waitcnt lgkmcnt(0)"
                 : RS_8_OUT(p), RS_8_OUT(q), "=&v"(scale[0]), "=&v"(scale[1]), "=&v"(scale[2]), "=&v"(scale[3])
                 : "v"(p_base + rp.at[0]), "v"(p_base + rp.at[1]), "v"(q_base + rq.at[0]), "v"(q_base + rq.at[1]),
                   "v"(scales)
                 : "memory");
#endif
}

__device__ __forceinline__ void read_q8(const Reader8 &r, unsigned base, unsigned scales, Operands8 &q,
                                        float (&scale)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile(RS_READ_8(0, 1, 2, 3, 4, 5, 6, 7, 12, 13) RS_READ_SCALES(8, 9, 10, 11, 14) "s_waitcnt lgkmcnt(0)"
                 : RS_8_OUT(q), "=&v"(scale[0]), "=&v"(scale[1]), "=&v"(scale[2]), "=&v"(scale[3])
                 : "v"(base + r.at[0]), "v"(base + r.at[1]), "v"(scales)
                 : "memory");
#endif
}

__global__ __launch_bounds__(kWideThreads) void wide_fp8_kernel(const ProductWork<fp8, bf16> w) {
    using OUT = bf16;
    __shared__ __align__(1024) char ring[kWideLds + 3 * kScaleBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = wave >> 2, p_wave = (wave & 3) * 64;
    const int num_rows = static_cast<int>(w.num_rows), p_tiles = (w.pn + kWide - 1) / kWide;
    const ResultTile t = rows_tile(w.offsets, w.experts, num_rows, kWide, p_tiles, w.clear, blockIdx.x);
    if (t.expert < 0) return;
    const int q0 = t.q * kWide, p0 = t.p * kWide;
    OUT *out = w.out;
    if (t.expert == w.experts) {
        clear_tile(out, w.out_stride, w.pn, RowTile{t.expert, t.q, t.rows}, kWide, num_rows, p0, kWide);
        return;
    }
    const int q_rows = t.rows.hi - t.rows.lo, c_n = w.cn;
    if (q0 >= q_rows || p0 >= w.pn) return;
    const fp8 *q = w.q + static_cast<size_t>(t.rows.lo) * w.q_stride;
    const fp8 *p = w.p + static_cast<size_t>(t.expert) * w.p_expert;
    out += static_cast<size_t>(t.rows.lo) * w.out_stride;
    const int left = q_rows - q0 < kWide ? q_rows - q0 : kWide;
    const int height = (left + 63) / 64 * 32, q_wave = group * height;

    constexpr int kStep = kStageBytes;
    static_assert(kStep == kScaleBlock);
    const int stages = (c_n + kStep - 1) / kStep;
    f32x4 acc[4][8];
#pragma unroll
    for (auto &a : acc) {
#pragma unroll
        for (auto &b : a) b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    Feeder<fp8, false, false> f0, f1;
    Feeder<fp8, false, true> fp;
    f0.set(q, w.q_stride, q_rows, c_n, q0, 0, height, wave, lane);
    f1.set(q, w.q_stride, q_rows, c_n, q0, 1, height, wave, lane);
    fp.set(p, w.p_stride, w.pn, c_n, p0, 0, 0, wave, lane);
    Reader8 rq, rp;
    rq.set(group * 64, lane);
    rp.set(p_wave, lane);
    const unsigned lds = lds_address(ring);
    const bool works = q0 + q_wave < q_rows && p0 + p_wave < w.pn;

    // Scales: waves 0 and 1 bring those of a group's 64 rows, a row a lane.
    const float *scale_base0 = uniform(w.q_scales + t.rows.lo + q0), *scale_base1 = scale_base0;
    const auto load_scales = [&](const float *&base, int first, int to) __attribute__((always_inline)) {
        const int row = (wave & 1) * height + first + lane;
        const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(base), 0, 0x7FFFFFFF, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)(ring + kWideLds + to + wave * 256), 4,
                                                 4 * (row < left ? row : left - 1), 0, 0, 0);
        base += w.num_rows;
    };
    // Of the matrix: one for the wave's 64 columns and a stage.
    const int p_block = p0 + p_wave < w.pn ? (p0 + p_wave) / kScaleBlock : 0;
    const size_t p_blocks = (static_cast<size_t>(w.pn) + kScaleBlock - 1) / kScaleBlock;
    const auto *p_scales = (const __attribute__((address_space(4))) float *)uniform(
        w.p_scales + (static_cast<size_t>(t.expert) * p_blocks + p_block) * stages);

    // Seven loads a wave: p, the first rows and their scales of stage s; three: the others.
    const auto load0 = [&](int s, char *to, int place) __attribute__((always_inline)) {
        load_scales(scale_base0, 0, place * kScaleBytes);
        fp.load(to, wave, lane, c_n - s * kStep);
        f0.load(to + kWideOperand, wave, lane, c_n - s * kStep);
    };
    const auto issue0 = [&](int s) __attribute__((always_inline)) {
        if (s < stages) load0(s, ring + s % 2 * kWideStage, s % 2);
    };
    const auto issue1 = [&](int s) __attribute__((always_inline)) {
        if (s >= stages) return;
        load_scales(scale_base1, 64, s % 2 * kScaleBytes + kScaleBytes / 2);
        f1.load(ring + s % 2 * kWideStage + kWideOperand * 3 / 2, wave, lane, c_n - s * kStep);
    };
    const auto arrived0 = [&](int s) __attribute__((always_inline)) {
        if (s + 1 < stages) {
            asm volatile("s_waitcnt vmcnt(10)" ::: "memory");
        } else if (s < stages) {
            asm volatile("s_waitcnt vmcnt(3)" ::: "memory");
        }
    };
    const auto arrived1 = [&](int s) __attribute__((always_inline)) {
        if (s + 1 < stages) {
            asm volatile("s_waitcnt vmcnt(10)" ::: "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
    };
    const auto barrier = []() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    Operands8 op, oq;
    float scale[4], p_scale = p_scales[0];
    f32x4 part[2][4] = {};
    float last_scale = 0.0f;
    const auto block = [&](auto j) __attribute__((always_inline)) {
        constexpr int J = decltype(j)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) part[J & 1][i] = mma16_fp8<kWhole8<OUT>>(op.f[i][0], op.f[i][1], oq.f[J][0], oq.f[J][1]);
    };
    const auto add = [&](auto half, auto j, float both) __attribute__((always_inline)) {
        constexpr int kHalf = decltype(half)::value, J = decltype(j)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                acc[i][4 * kHalf + J][r] = __builtin_fmaf(part[J & 1][i][r], both, acc[i][4 * kHalf + J][r]);
            }
        }
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    constexpr std::integral_constant<int, 3> k3{};
    // Multiplies rows 64 HALF .. of the group, 16 times BLOCKS (2 or 4), with the
    // operands read last, and adds all but the last 16 rows' results, which finish() does
    // beside the other group's products.
    const auto multiply = [&](auto half, auto blocks) __attribute__((always_inline)) {
        __builtin_amdgcn_s_setprio(1);
        block(k0), block(k1), add(half, k0, scale[0] * p_scale);
        if constexpr (decltype(blocks)::value == 4) {
            block(k2), add(half, k1, scale[1] * p_scale), block(k3), add(half, k2, scale[2] * p_scale);
        }
        last_scale = scale[decltype(blocks)::value - 1] * p_scale;
        // An instruction for the matrix unit, then four for the others.
        __builtin_amdgcn_sched_group_barrier(0x8, 5, 0);
#pragma unroll
        for (int i = 0; i < 4 * decltype(blocks)::value - 5; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        }
        __builtin_amdgcn_s_setprio(0);
    };
    const auto finish = [&](auto half, auto blocks) __attribute__((always_inline)) {
        add(half, std::integral_constant<int, decltype(blocks)::value - 1>{}, last_scale);
    };
    constexpr std::integral_constant<int, 4> k4{};
    const unsigned scales_at = lds + kWideLds + static_cast<unsigned>(group * 64 + (lane & 15)) * 4;
    // Slots as in wide_product_kernel.
    const auto tall = [&](auto others) __attribute__((always_inline)) {
        issue0(0);
        issue1(0);
        issue0(1);
        if (stages > 1) {
            asm volatile("s_waitcnt vmcnt(7)" ::: "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        barrier();
        if (group == 1) barrier();
#pragma nounroll
        for (int s = 0; s < stages; ++s) {
            const unsigned at = lds + static_cast<unsigned>(s % 2) * kWideStage;
            const unsigned of = scales_at + static_cast<unsigned>(s % 2) * kScaleBytes;
            if (works) {
                read_pq8(rq, rp, at + kWideOperand, at, of, oq, op, scale);
                finish(k1, others);  // of the stage before
            }
            issue1(s + 1);
            if (group == 1) arrived1(s);
            barrier();
            if (works) multiply(k0, k4);
            if (group == 0) arrived1(s);
            barrier();
            if (works) {
                read_q8(rq, at + kWideOperand * 3 / 2, of + kScaleBytes / 2, oq, scale);
                finish(k0, k4);
            }
            issue0(s + 2);
            if (group == 1) arrived0(s + 1);
            barrier();
            if (works) multiply(k1, others);
            p_scale = p_scales[s + 1 < stages ? s + 1 : s];
            if (group == 0) arrived0(s + 1);
            if (s + 1 < stages || group == 0) barrier();
        }
        if (works) finish(k1, others);
    };
    const auto flat = [&](auto rows) __attribute__((always_inline)) {
        const auto issue = [&](int s, unsigned place) __attribute__((always_inline)) {
            if (s < stages) load0(s, ring + place * kFlatStage, static_cast<int>(place));
        };
        const auto arrived = [&](int s) __attribute__((always_inline)) {
            if (s + 1 < stages) {
                asm volatile("s_waitcnt vmcnt(7)" ::: "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
        };
        issue(0, 0);
        issue(1, 1);
        arrived(0);
        if (group == 1) issue(2, 2);
        barrier();
        if (group == 1) barrier();
        unsigned place = 0;
#pragma nounroll
        for (int s = 0; s < stages; ++s) {
            const unsigned at = lds + place * kFlatStage, before = place == 0 ? 2 : place - 1;
            if (works) {
                read_pq8(rq, rp, at + kWideOperand, at, scales_at + place * kScaleBytes, oq, op, scale);
                finish(k0, rows);
            }
            if (group == 0) {
                issue(s + 2, before);
            } else {
                arrived(s + 1);
            }
            barrier();
            if (group == 1) issue(s + 3, place);
            if (works) multiply(k0, rows);
            p_scale = p_scales[s + 1 < stages ? s + 1 : s];
            if (group == 0) arrived(s + 1);
            if (s + 1 < stages || group == 0) barrier();
            place = place == 2 ? 0 : place + 1;
        }
        if (works) finish(k0, rows);
    };
    if (height == 128) {
        tall(k4);
    } else if (height == 96) {
        tall(k2);
    } else if (height == 64) {
        flat(k4);
    } else {
        flat(k2);
    }

    char *mine = ring + wave * 16384;
    typedef OUT t4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = 16 * j + (lane & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = static_cast<OUT>(acc[i][j][r]);
            const int chunk = 2 * i + (lane >> 5);
            *reinterpret_cast<t4 *>(mine + result_at(row, chunk) + (lane >> 4 & 1) * 8) = v;
        }
    }
    wave_exchange();
    rows_from_lds(mine, out, w.out_stride, height, q0 + q_wave, q_rows, p0 + p_wave, w.pn, lane);
}

}  // namespace rs
