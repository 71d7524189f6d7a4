// products.hip -- C ABI of the experts' own work (matrix products of sorted
// rows, rows in 8 bits, gated rows): argument checks and launches.
#include <algorithm>
#include <cmath>

#include "gates.hpp"
#include "launch.hpp"
#include "products.hpp"
#include "products_few.hpp"
#include "products_split.hpp"
#include "products_wide.hpp"

// Named here, as the host's pass does not emit all of those that only calls within
// generic lambdas name.
#define RS_WIDE(T)                                                                                          \
    template __global__ void rs::wide_product_kernel<T, false, false, false>(const rs::ProductWork<T, T>); \
    template __global__ void rs::wide_product_kernel<T, false, false, true>(const rs::ProductWork<T, T>);  \
    template __global__ void rs::wide_product_kernel<T, true, true, true>(const rs::ProductWork<T, T>);
RS_WIDE(rs::f16)
RS_WIDE(rs::bf16)
#undef RS_WIDE

namespace {

int g_product_kernel = 0;  // rs_prof_product_kernel: 0 automatic, else an rs_product_kernel where it can serve

constexpr int kMaxWidth = RS_MAX_ROW_WIDTH;
constexpr size_t kMaxExpertStride = size_t{1} << 50;

bool good_groups(const int32_t *offsets, int experts, size_t num_rows) {
    if (experts < 1 || experts > RS_MAX_EXPERTS || num_rows > RS_MAX_PRODUCT_ROWS) return false;
    return offsets == nullptr ? experts == 1 : aligned(offsets, 4);
}

Span span_offsets(const int32_t *offsets, int experts) {
    return span_of(offsets, offsets ? 4 * (static_cast<size_t>(experts) + 1) : 0);
}

// Matrices [experts][rows][width], read.
struct Matrices {
    const void *p;
    int experts, rows, width;
    size_t stride, expert, elem;

    bool good() const {
        return ::good(p, 1, elem) && rows >= 1 && rows <= kMaxWidth && width >= 1 && width <= kMaxWidth &&
               stride <= kMaxStride && expert <= kMaxExpertStride;
    }
    Span span() const {
        const size_t last = static_cast<size_t>(experts - 1) * expert + static_cast<size_t>(rows - 1) * stride;
        return span_of(p, (last + static_cast<size_t>(width)) * elem);
    }
};

size_t scale_blocks(int width) { return (static_cast<size_t>(width) + rs::kScaleBlock - 1) / rs::kScaleBlock; }

bool addressable(Span s) { return s.lo <= s.hi && s.hi - s.lo < (size_t{1} << 62); }

size_t align_to(size_t x, size_t by) { return (x + by - 1) / by * by; }

size_t parts(size_t x, size_t by) { return (x + by - 1) / by; }

// Workgroups of a launch whose tiles may be many: below 2^32 threads, all that a launch
// counts to.
constexpr size_t kMostTiles = size_t{1} << 22;
static_assert(kMostTiles * rs::kWideThreads < size_t{1} << 32);

// Whether the wide kernel can take an operand: its 16-byte chunks are aligned, a
// tile spans less than 2^31 bytes, and a row has a chunk (across: whole ones).
bool feeds(const void *p, size_t stride, size_t expert, int width, bool across, size_t elem) {
    const size_t chunk = 16 / elem;
    return aligned(p, 16) && stride % chunk == 0 && expert % chunk == 0 && stride <= (size_t{1} << 22) &&
           width >= static_cast<int>(chunk) && (!across || static_cast<size_t>(width) % chunk == 0);
}

// Whether both operands' rows begin at 16 bytes.
template <class T, class OUT>
bool aligned_rows(const rs::ProductWork<T, OUT> &w) {
    constexpr size_t kChunk = 16 / sizeof(T);
    return aligned(w.q, 16) && aligned(w.p, 16) && w.q_stride % kChunk == 0 && w.p_stride % kChunk == 0 &&
           w.p_expert % kChunk == 0;
}

// ---------------------------------------------------------------------------
// Which kernel takes a product, by estimates of their times in us (with 4 to 6 for the
// launch and its beginning).  The experts are taken to have equally many rows.
//
// Tiles go round the 256 CUs: the wide kernel's stage of 128 bytes of c takes 0.55 us, as
// long as its loads are on their way, and more for a tile full of rows; but
// memory gives no more than 6 TB/s; a tile of the weights' gradient, whose stages are few, begins
// and ends in 6 (3.5 for two square ones), one of 8 bits in 4.  The kernel for few rows reads weights at 5 to
// 6 TB/s, and its rows again for each of its strips, at 25.4 GB/s a CU, or 4.3 if they do not
// begin at 16 bytes (in float32 it multiplies at 75 TFLOP/s).  Square tiles take 0.85 us for
// 128 bytes of c, 1.25 if rows do not begin at 16 bytes, and 1.5 if two share
// every CU, in 8 bits 1.4 and 2.6; of 64 x 64 in float32 1, and 0.52 of a CU's time.  Tiles whose
// contraction is split take 1.4 us for eight times 128 bytes on half of the CUs and 1.75 on all, in 8 bits
// 2.2, 2.6 and, if they are many, 3.3, where rows do not begin at 16 bytes 1.9 and 3.  Whole sums of
// 8-bit operands take 1.1 to 1.3 times as long, in few rows 1.5 us a round more.
// Rows of no expert, which only the offsets on the device tell, count as if they had one.
// Measured, in us, wide / few rows / square / split (bfloat16, rows x experts x out x in):
// 8 of 64 x 2048 x 2048 23 / 12 / 27 / 14, 512 of 64 x 4096 x 4096 369 / 400 / 384 / 374, 16 of one x
// 8192 x 8192 77 / 28 / 92 / 30, 128 of one 94 / 88 / 93 / 34, 256 of one 155 / 174 / 94 / 63,
// 300 of 16 x 2048 x 2048 23 / 27 / 29 / 27, 512 of 8 x 1024 x 1024 15 / 9 / 14 / 8, 2048 of 8 25 / 25 / 15 / 16,
// 1000 of 7 x 1001 x 1537 - / 77 / 33 / 26, 40 of 7 - / 17 / 32 / 14, 5003 of 7 - / 302 / 45 / 80,
// 64 of one x 1024 x 8192 84 / 37 / 81 / 28, 256 of one x 4096 x 4096 82 / 47 / 50 / 20, 1024 of one 83 / 169 / 56 / 70;
// rows' gradient, 128 of one x 4096 x 4096 49 / - / 51 / 18; weights' gradient, 8192 of one x 1024 x 1024
// 169 / - / 96 / 32, 9076 of 2 x 128 x 512 55 / - / 56 / 17, 4096 of 8 x 1024 x 1024 19 / - / 17 / 39, 16384 of
// 64 x 1024 x 2048 125 / - / 163 / 476; e4m3, and with whole sums, 256 of 128 x 2048 x 4096 181 / 171 / 283 / 272, - / 212 / 341 / 285,
// 128 of one x 4096 x 8192 66 / 27 / 98 / 19, - / 33 / 100 / 24, 4000 of 8 x 1024 x 2048 35 / 68 / 27 / 32, - / 78 / 28 / 38,
// 25412 of 89 x 321 x 640 34 / - / 30 / 65, - / - / 32 / 70, 512 of one x 7168 x 4096 63 / 101 / 54 / 46, - / 115 / 54 / 54.
// The choice is off where two are close, and by more for some decoding batches: 16 of 64 x 2048 x 2088 go to
// the wide kernel, 29 / 21 / 32 / 25.
// ---------------------------------------------------------------------------
constexpr double kTwoStrips = 512;  // workgroups of few_rows_kernel, of one strip, from which on they take two

struct Estimate {
    double rows_each, experts_used, weight_bytes, stages, pn;
    bool bytes, words;  // operands of 8, of 32 bits
    bool whole;         // of 8 bits, with whole sums
    bool apart;         // rows that do not begin at 16 bytes
    bool ragged_c;

    template <class T, class OUT>
    Estimate(const rs::ProductWork<T, OUT> &w, bool of_weights)
        : pn(w.pn), bytes(sizeof(T) == 1), words(sizeof(T) == 4), whole(bytes && rs::kWhole8<OUT>),
          apart(!aligned_rows(w)), ragged_c(of_weights) {
        const double n = static_cast<double>(w.num_rows), e = static_cast<double>(w.experts);
        if (ragged_c) {
            experts_used = e, rows_each = w.qn;
            weight_bytes = e * w.pn * w.qn * static_cast<double>(sizeof(T));
            stages = std::ceil(n / e * static_cast<double>(sizeof(T)) / 128);
            return;
        }
        experts_used = std::max(1.0, e * (1.0 - std::exp(-n / e)));  // by rows that choose at random
        rows_each = n / experts_used;
        weight_bytes = experts_used * w.pn * w.cn * static_cast<double>(sizeof(T));
        stages = static_cast<double>(parts(static_cast<size_t>(w.cn) * sizeof(T), 128));
    }
    double tiles(double height, double width) const {
        return experts_used * std::ceil(rows_each / height) * std::ceil(pn / width);
    }
    double wide() const {
        const double t = tiles(rs::kWide, rs::kWide);
        const double full = bytes ? (t > 128 ? 1.45 : 1.0) : t > 128 ? 1.1 : 0.65;
        const double stage = 0.55 + full * std::min(1.0, rows_each / rs::kWide), ends = ragged_c ? 6 : bytes ? 4 : 0;
        return 6 + std::max(std::ceil(t / 256) * (stages * stage + ends), weight_bytes / (bytes ? 5.5e6 : 6e6));
    }
    int few_rows() const { return rows_each <= 12 ? 1 : rows_each <= 28 ? 2 : 4; }  // 16 of them each
    double few() const {
        const double weights = weight_bytes / (whole ? 5.2e6 : bytes ? 6e6 : 5.2e6);
        const int height = 16 * few_rows();
        const double groups = tiles(height, 16) >= kTwoStrips ? tiles(height, 32) : tiles(height, 16);
        const double taken = (std::min(rows_each, 1.0 * height) + height) / 2;  // (loads of rows that do not exist count half)
        const double rounds = std::ceil(groups / 256);
        double rows = rounds * taken * stages * 128 / (apart ? 4.3e3 : 25.4e3);
        if (whole) rows = 1.3 * rows + 1.5 * (rounds - 1);
        if (words) rows = std::max(rows, experts_used * rows_each * stages * std::ceil(pn / 32) * 2.0 * 32 * 32 / 75e6);
        return 4 + std::max(weights, rows) + 0.25 * std::min(weights, rows);
    }
    double square() const {
        const double t = words ? tiles(64, 64) : tiles(128, 128);
        const double alone = whole ? 1.5 : bytes ? 1.4 : apart ? 1.25 : 0.85, two = whole ? 3.0 : bytes ? 2.6 : 1.5;
        const double step = words ? std::max(1.0, 0.52 * t / 256) : t <= 256 ? alone : two * std::ceil(t / 512);
        const double ends = ragged_c && t > 256 ? 3.5 * std::ceil(t / 512) : 0;
        return 4 + std::max(stages * step + ends, weight_bytes / 3.5e6);
    }
    double split() const {
        const double t = tiles(rs::kSplitSide, rs::kSplitSide);
        const double some = whole ? 2.6 : apart ? 1.9 : bytes ? 2.2 : 1.4;
        const double all = apart ? 3.0 : whole ? 2.9 : bytes ? 2.6 : 1.75;
        const double step = t <= 128 ? some : bytes && t > 512 ? (whole ? 3.6 : 3.3) : all;
        return 4 + std::max(std::ceil(t / 256) * (std::ceil(stages / rs::kSplitWaves) * step + 2), weight_bytes / 3.5e6);
    }
};

// Enqueues few_rows_kernel: as few rows as the experts have on average fill the
// matrix instruction's 16 columns up; two strips a workgroup of four waves where
// every CU has a workgroup then, or else one strip and more waves for the
// contraction: one row, 4096 x 4096 bfloat16, 11.8 us with two strips and 4 waves, 8.7 with one
// and 16; 16 rows, 8192 x 8192, 35 and 39.
template <class T, class OUT>
bool launch_few(const rs::ProductWork<T, OUT> &w, const Estimate &e, hipStream_t stream) {
    const auto with_rows = [&](auto rows) {
        constexpr int R = decltype(rows)::value;
        const size_t q_tiles = w.num_rows / (16 * R) + std::min<size_t>(w.num_rows, static_cast<size_t>(w.experts)) + 1;
        const auto go = [&](auto kernel, int waves, int strips_each, size_t p_tiles) {
            return launch_kernel(RS_KERNEL_PRODUCT, stream, [&] {
                run_kernel(kernel, static_cast<unsigned>(q_tiles * p_tiles), 64 * waves, stream, w);
            }, RS_PRODUCT_FEW + 16 * R + 256 * strips_each);
        };
        const size_t strips = parts(static_cast<size_t>(w.pn), 16);
        const double groups = e.tiles(16 * R, 16);
        if (groups >= kTwoStrips) return go(rs::few_rows_kernel<T, OUT, 4, 2, R>, 4, 2, parts(strips, 2));
        constexpr int kWaves = R == 4 ? 8 : 16;  // (16 would have registers for a step at a time)
        return go(rs::few_rows_kernel<T, OUT, kWaves, 1, R>, kWaves, 1, strips);
    };
    if (e.few_rows() == 1) return with_rows(IntC<1>{});
    if (e.few_rows() == 2) return with_rows(IntC<2>{});
    return with_rows(IntC<4>{});
}

// Enqueues the product of w, whose results are q by p (RAGGED_C: of each expert).
template <class T, class OUT, bool RAGGED_C, bool Q_ACROSS, bool P_ACROSS>
bool launch_product(const rs::ProductWork<T, OUT> &w, hipStream_t stream) {
    const int least = std::min(Q_ACROSS ? w.qn : w.cn, P_ACROSS ? w.pn : w.cn);  // width of a row
    // Tiles of `side` results, or of rows of none, at most.  Each expert's last tile may be a part, and
    // so may that of the rows of none; eighths of either go to an XCD.
    const auto jobs_of = [&](size_t side) {
        const size_t p_tiles = parts(static_cast<size_t>(w.pn), side);
        return RAGGED_C
            ? align_to(parts(static_cast<size_t>(w.qn), side) * p_tiles, rs::kXcds) * static_cast<size_t>(w.experts)
            : align_to((w.num_rows / side + std::min<size_t>(w.num_rows, static_cast<size_t>(w.experts)) + 1) * p_tiles,
                       rs::kXcds) + rs::kXcds;
    };
    const Estimate e(w, RAGGED_C);
    constexpr double kNever = 1e30;
    const bool chunks = least >= static_cast<int>(16 / sizeof(T));  // a row has 16 bytes
    double square = e.square(), wide = kNever, few = kNever, split = kNever;
    const auto force = [](double &time, int kernel) {
        if (g_product_kernel == kernel && time != kNever) time = 0;
    };
    if constexpr (sizeof(T) <= 2) {
        // (Below a stage of rows, what counts for the weights' gradient is that it is written from many CUs.)
        if (jobs_of(rs::kWide) <= kMostTiles && feeds(w.q, w.q_stride, 0, Q_ACROSS ? w.qn : w.cn, Q_ACROSS, sizeof(T)) &&
            feeds(w.p, w.p_stride, w.p_expert, P_ACROSS ? w.pn : w.cn, P_ACROSS, sizeof(T)) &&
            (!RAGGED_C || w.num_rows >= 64 * static_cast<size_t>(w.experts)) && !(sizeof(T) == 1 && rs::kWhole8<OUT>)) {
            wide = e.wide();
        }
        // (In float32 a CU's matrix units are busy with one tile of 64 x 64.)
        if (chunks && jobs_of(rs::kSplitSide) <= kMostTiles) split = e.split();
    }
    force(square, RS_PRODUCT_SQUARE), force(wide, RS_PRODUCT_WIDE), force(split, RS_PRODUCT_SPLIT);
    if constexpr (!RAGGED_C && !P_ACROSS) {
        // (A strip and up to 1024 threads, or where strips are many two and 256.)
        const size_t strips = parts(static_cast<size_t>(w.pn), 16) *
            (w.num_rows / 16 + std::min<size_t>(w.num_rows, static_cast<size_t>(w.experts)) + 1);
        if (chunks && w.num_rows <= 65536 && strips <= 4 * kMostTiles) few = e.few();
        force(few, RS_PRODUCT_FEW);
        if (few <= std::min({wide, square, split})) return launch_few(w, e, stream);
    }
    const auto launch = [&](auto kernel, int which, size_t grid, int threads, const auto &work) {
        return launch_kernel(RS_KERNEL_PRODUCT, stream,
                             [&] { run_kernel(kernel, static_cast<unsigned>(grid), threads, stream, work); }, which);
    };
    if constexpr (sizeof(T) <= 2) {
        if (wide <= std::min(square, split)) {
            if constexpr (sizeof(T) == 1 && rs::kWhole8<OUT>) {
                return false;  // (not estimated)
            } else if constexpr (sizeof(T) == 1) {
                return launch(rs::wide_fp8_kernel, RS_PRODUCT_WIDE, jobs_of(rs::kWide), rs::kWideThreads, w);
            } else {
                return launch(rs::wide_product_kernel<T, RAGGED_C, Q_ACROSS, P_ACROSS>, RS_PRODUCT_WIDE,
                              jobs_of(rs::kWide), rs::kWideThreads, w);
            }
        }
        if (split < square) {
            return launch(rs::split_kernel<T, OUT, RAGGED_C, Q_ACROSS, P_ACROSS>, RS_PRODUCT_SPLIT,
                          jobs_of(rs::kSplitSide), 64 * rs::kSplitWaves, w);
        }
    }
    const size_t jobs = jobs_of(rs::kSquare<T>);
    if (jobs > size_t{1} << 31) return false;  // (whose results no memory holds)
    rs::ProductWork<T, OUT> work = w;
    work.jobs = static_cast<unsigned>(jobs);
    const auto go = [&](auto kernel) { return launch(kernel, RS_PRODUCT_SQUARE, std::min(jobs, kMostTiles), 256, work); };
    if (!chunks) return go(rs::product_kernel<T, OUT, RAGGED_C, Q_ACROSS, P_ACROSS, 1, true>);
    // (Rows that take less than two steps are not worth the registers of a second, and beside
    // whole sums of 8-bit operands there are none: registers spill: twice the time.)
    constexpr bool kOne = sizeof(T) == 1 && rs::kWhole8<OUT>;
    if (sizeof(T) < 4 && (kOne || !aligned_rows(w) || (RAGGED_C && w.num_rows < 128 * static_cast<size_t>(w.experts)))) {
        return go(rs::product_kernel<T, OUT, RAGGED_C, Q_ACROSS, P_ACROSS, 1, false>);
    }
    if constexpr (!kOne) return go(rs::product_kernel<T, OUT, RAGGED_C, Q_ACROSS, P_ACROSS, 2, false>);
    return false;
}

rs::Divider divider(size_t by) {
    unsigned up = 0;
    while ((size_t{1} << up) < by) ++up;
    return {static_cast<uint32_t>(((uint64_t{1} << (31 + up)) + by - 1) / by), 31 + up};
}

template <class F>
bool with_act(int act, F &&f) {
    return act == RS_ACT_GELU ? f(IntC<rs::kActGelu>{}) : f(IntC<rs::kActSilu>{});
}

// Calls f(IntC of a rs::Row) for rows of `width` elements, `vec` of them 16 bytes.
template <class F>
bool with_row(int width, int vec, F &&f) {
    if (width < vec) return f(IntC<rs::kNarrowRow>{});
    return width % 8 == 0 ? f(IntC<rs::kWholeRow>{}) : f(IntC<rs::kRaggedRow>{});
}

bool good_gate(int dtype, int act, int width) {
    return dtype_bytes(dtype) != 0 && (act == RS_ACT_SILU || act == RS_ACT_GELU) && width >= 1 && width <= kMaxWidth / 2;
}

// Enqueues h = act(a) b of rows, or its gradient if grad is given.
rs_status gate_rows(const void *grad, size_t grad_stride, const void *rows, int dtype, size_t num_rows, int width,
                    size_t rows_stride, const int32_t *offsets, int experts, int act, void *out, size_t out_stride,
                    int all, bool backward, hipStream_t stream) {
    if (!good_gate(dtype, act, width) || !good_groups(offsets, experts, num_rows)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype));
    const int out_width = backward ? 2 * width : width;
    if (!good_rows(rows, num_rows, 2 * width, rows_stride, elem, false) ||
        !good_rows(out, num_rows, out_width, out_stride, elem, true) ||
        (backward && !good_rows(grad, num_rows, width, grad_stride, elem, false))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const auto wide = static_cast<size_t>(width);
    const Span spans[] = {span_of(out, span_bytes(num_rows, static_cast<size_t>(out_width), out_stride, elem)),
                          span_of(rows, span_bytes(num_rows, 2 * wide, rows_stride, elem)),
                          span_of(grad, backward ? span_bytes(num_rows, wide, grad_stride, elem) : 0),
                          span_offsets(offsets, experts)};
    if (!disjoint(spans, 1, 4)) return RS_ERROR_INVALID_VALUE;
    if (num_rows == 0) return RS_SUCCESS;
    rs::GateWork w{};
    w.rows = rows, w.grad = grad, w.out = out;
    w.rows_stride = rows_stride, w.grad_stride = grad_stride, w.out_stride = out_stride;
    w.offsets = offsets, w.experts = experts, w.num_rows = num_rows, w.width = width, w.clear = all != 0;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_act(act, [&](auto a) {
            constexpr int kAct = decltype(a)::value;
            const auto go = [&](auto kernel, int v) {
                w.chunks = (width + v - 1) / v;
                const size_t units = num_rows * static_cast<size_t>(w.chunks);
                const unsigned grid = grid_for(units, rs::kGateBlock, kMaxGrid);
                return launch_kernel(RS_KERNEL_GATE, stream, [&] {
                    run_kernel(kernel, grid, rs::kGateBlock, stream, w, divider(static_cast<size_t>(w.chunks)));
                });
            };
            constexpr int V = rs::kVec<T>;
            if (width < V) {
                return backward ? go(rs::gate_kernel<T, 1, kAct, true>, 1) : go(rs::gate_kernel<T, 1, kAct, false>, 1);
            }
            return backward ? go(rs::gate_kernel<T, V, kAct, true>, V) : go(rs::gate_kernel<T, V, kAct, false>, V);
        });
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

// Enqueues rows (gate: act(a) b of them) in 8 bits with their scales.
rs_status quantize_rows(const void *rows, int dtype, size_t num_rows, int width, size_t rows_stride,
                        const int32_t *offsets, int experts, bool gate, int act, uint8_t *out, size_t out_stride,
                        float *scales, int all, hipStream_t stream) {
    if (gate ? !good_gate(dtype, act, width) : dtype_bytes(dtype) == 0 || width < 1 || width > kMaxWidth) {
        return RS_ERROR_INVALID_VALUE;
    }
    if (!good_groups(offsets, experts, num_rows)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), blocks = scale_blocks(width);
    const int in_width = gate ? 2 * width : width;
    if (!good_rows(rows, num_rows, in_width, rows_stride, elem, false) ||
        !good_rows(out, num_rows, width, out_stride, 1, true) || !good(scales, num_rows, 4)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const Span spans[] = {span_of(out, span_bytes(num_rows, static_cast<size_t>(width), out_stride, 1)),
                          span_of(scales, num_rows * blocks * 4),
                          span_of(rows, span_bytes(num_rows, static_cast<size_t>(in_width), rows_stride, elem)),
                          span_offsets(offsets, experts)};
    if (!disjoint(spans, 2, 4)) return RS_ERROR_INVALID_VALUE;
    if (num_rows == 0) return RS_SUCCESS;
    rs::GateWork w{};
    w.rows = rows, w.out = out, w.scales = scales, w.rows_stride = rows_stride, w.out_stride = out_stride;
    w.offsets = offsets, w.experts = experts, w.num_rows = num_rows, w.width = width, w.clear = all != 0;
    const int per_group = gate ? rs::kQuantizeBlocks<true> : rs::kQuantizeBlocks<false>;
    const dim3 grid(static_cast<unsigned>(parts(blocks, static_cast<size_t>(per_group))),
                    static_cast<unsigned>(std::min<size_t>(parts(num_rows, 16), 65535)));
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        const auto go = [&](auto kernel) {
            return launch_kernel(RS_KERNEL_QUANTIZE, stream,
                                 [&] { run_kernel(kernel, grid, rs::kGateBlock, stream, w); });
        };
        return with_row(width, rs::kVec<T>, [&](auto row) {
            constexpr int kRow = decltype(row)::value;
            if (!gate) return go(rs::quantize_rows_kernel<T, 0, false, kRow>);
            return with_act(act, [&](auto a) { return go(rs::quantize_rows_kernel<T, decltype(a)::value, true, kRow>); });
        });
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

}  // namespace

extern "C" {

int rs_prof_product_kernel(int kernel) {
    const int prev = g_product_kernel;
    g_product_kernel = kernel >= RS_PRODUCT_SQUARE && kernel <= RS_PRODUCT_WIDE ? kernel : 0;
    return prev;
}

rs_status rs_expert_products(const void *rows, int dtype, size_t num_rows, int in_width, size_t rows_stride,
                             const int32_t *offsets, int experts, const void *weights, int out_width,
                             size_t weights_stride, size_t weights_expert, void *out, size_t out_stride, int all,
                             hipStream_t stream) {
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype));
    if (elem == 0 || !good_groups(offsets, experts, num_rows)) return RS_ERROR_INVALID_VALUE;
    const Matrices m{weights, experts, out_width, in_width, weights_stride, weights_expert, elem};
    if (!m.good() || !good_rows(rows, num_rows, in_width, rows_stride, elem, false) ||
        !good_rows(out, num_rows, out_width, out_stride, elem, true)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const Span spans[] = {span_of(out, span_bytes(num_rows, static_cast<size_t>(out_width), out_stride, elem)),
                          span_of(rows, span_bytes(num_rows, static_cast<size_t>(in_width), rows_stride, elem)), m.span(),
                          span_offsets(offsets, experts)};
    if (!addressable(spans[2]) || !disjoint(spans, 1, 4)) return RS_ERROR_INVALID_VALUE;
    if (num_rows == 0) return RS_SUCCESS;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        rs::ProductWork<T, T> w{};
        w.q = static_cast<const T *>(rows), w.q_stride = rows_stride;
        w.p = static_cast<const T *>(weights), w.p_stride = weights_stride, w.p_expert = weights_expert;
        w.out = static_cast<T *>(out), w.out_stride = out_stride;
        w.offsets = offsets, w.experts = experts, w.num_rows = num_rows;
        w.pn = out_width, w.cn = in_width, w.clear = all != 0;
        return launch_product<T, T, false, false, false>(w, stream);
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_expert_products_backward(const void *grad, int dtype, size_t num_rows, int out_width, size_t grad_stride,
                                      const int32_t *offsets, int experts, const void *weights, size_t weights_stride,
                                      size_t weights_expert, const void *rows, size_t rows_stride, int in_width,
                                      void *grad_rows, size_t grad_rows_stride, void *grad_weights, int all,
                                      hipStream_t stream) {
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype));
    if (elem == 0 || !good_groups(offsets, experts, num_rows)) return RS_ERROR_INVALID_VALUE;
    const auto wide_in = static_cast<size_t>(in_width), wide_out = static_cast<size_t>(out_width);
    if (in_width < 1 || in_width > kMaxWidth || out_width < 1 || out_width > kMaxWidth ||
        !good_rows(grad, num_rows, out_width, grad_stride, elem, false)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const bool to_rows = grad_rows != nullptr, to_weights = grad_weights != nullptr;
    const Matrices m{weights, experts, out_width, in_width, weights_stride, weights_expert, elem};
    if (to_rows && (!m.good() || !good_rows(grad_rows, num_rows, in_width, grad_rows_stride, elem, true))) {
        return RS_ERROR_INVALID_VALUE;
    }
    if (to_weights && (!aligned(grad_weights, elem) || !good_rows(rows, num_rows, in_width, rows_stride, elem, false))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const size_t matrix = wide_in * wide_out;
    const Span spans[] = {span_of(grad_rows, to_rows ? span_bytes(num_rows, wide_in, grad_rows_stride, elem) : 0),
                          span_of(grad_weights, to_weights ? static_cast<size_t>(experts) * matrix * elem : 0),
                          span_of(grad, span_bytes(num_rows, wide_out, grad_stride, elem)),
                          to_rows ? m.span() : span_of(weights, 0),
                          span_of(rows, to_weights ? span_bytes(num_rows, wide_in, rows_stride, elem) : 0),
                          span_offsets(offsets, experts)};
    if (!addressable(spans[1]) || !addressable(spans[3]) || !disjoint(spans, 2, 6)) return RS_ERROR_INVALID_VALUE;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        rs::ProductWork<T, T> w{};
        w.q = static_cast<const T *>(grad), w.q_stride = grad_stride;
        w.offsets = offsets, w.experts = experts, w.num_rows = num_rows, w.pn = in_width;
        if (to_rows && num_rows != 0) {
            w.p = static_cast<const T *>(weights), w.p_stride = weights_stride, w.p_expert = weights_expert;
            w.out = static_cast<T *>(grad_rows), w.out_stride = grad_rows_stride;
            w.cn = out_width, w.clear = all != 0;
            if (!launch_product<T, T, false, false, true>(w, stream)) return false;
        }
        if (!to_weights) return true;
        w.p = static_cast<const T *>(rows), w.p_stride = rows_stride, w.p_expert = 0;
        w.out = static_cast<T *>(grad_weights), w.out_stride = wide_in, w.out_expert = matrix;
        w.qn = out_width, w.cn = 0;
        return launch_product<T, T, true, true, true>(w, stream);
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_expert_products_fp8(const uint8_t *rows, const float *row_scales, size_t num_rows, int in_width,
                                 size_t rows_stride, const int32_t *offsets, int experts, const uint8_t *weights,
                                 const float *weight_scales, int out_width, size_t weights_stride,
                                 size_t weights_expert, void *out, int dtype, size_t out_stride, int all,
                                 hipStream_t stream) {
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype));
    if (elem == 0 || !good_groups(offsets, experts, num_rows)) return RS_ERROR_INVALID_VALUE;
    const Matrices m{weights, experts, out_width, in_width, weights_stride, weights_expert, 1};
    if (!m.good() || !good_rows(rows, num_rows, in_width, rows_stride, 1, false) || !good(row_scales, num_rows, 4) ||
        !good(weight_scales, 1, 4) || !good_rows(out, num_rows, out_width, out_stride, elem, true)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const size_t blocks = scale_blocks(in_width), out_blocks = scale_blocks(out_width);
    const Span spans[] = {span_of(out, span_bytes(num_rows, static_cast<size_t>(out_width), out_stride, elem)),
                          span_of(rows, span_bytes(num_rows, static_cast<size_t>(in_width), rows_stride, 1)), m.span(),
                          span_of(row_scales, num_rows * blocks * 4),
                          span_of(weight_scales, static_cast<size_t>(experts) * blocks * out_blocks * 4),
                          span_offsets(offsets, experts)};
    if (!addressable(spans[2]) || !disjoint(spans, 1, 6)) return RS_ERROR_INVALID_VALUE;
    if (num_rows == 0) return RS_SUCCESS;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using OUT = decltype(zero);
        rs::ProductWork<rs::fp8, OUT> w{};
        w.q = reinterpret_cast<const rs::fp8 *>(rows), w.q_stride = rows_stride, w.q_scales = row_scales;
        w.p = reinterpret_cast<const rs::fp8 *>(weights), w.p_stride = weights_stride, w.p_expert = weights_expert;
        w.p_scales = weight_scales;
        w.out = static_cast<OUT *>(out), w.out_stride = out_stride;
        w.offsets = offsets, w.experts = experts, w.num_rows = num_rows;
        w.pn = out_width, w.cn = in_width, w.clear = all != 0;
        return launch_product<rs::fp8, OUT, false, false, false>(w, stream);
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_quantize_rows(const void *rows, int dtype, size_t num_rows, int width, size_t rows_stride,
                           const int32_t *offsets, int experts, uint8_t *out, size_t out_stride, float *scales, int all,
                           hipStream_t stream) {
    return quantize_rows(rows, dtype, num_rows, width, rows_stride, offsets, experts, false, RS_ACT_SILU, out, out_stride,
                         scales, all, stream);
}

rs_status rs_quantize_weights(const void *weights, int dtype, int experts, int out_width, int in_width,
                              size_t weights_stride, size_t weights_expert, uint8_t *out, float *scales,
                              hipStream_t stream) {
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype));
    if (elem == 0 || experts < 1 || experts > RS_MAX_EXPERTS) return RS_ERROR_INVALID_VALUE;
    const Matrices m{weights, experts, out_width, in_width, weights_stride, weights_expert, elem};
    if (!m.good() || !good(out, 1, 1) || !good(scales, 1, 4)) return RS_ERROR_INVALID_VALUE;
    const size_t e = static_cast<size_t>(experts);
    const size_t blocks = e * scale_blocks(out_width) * scale_blocks(in_width);
    const Span spans[] = {span_of(out, e * static_cast<size_t>(out_width) * static_cast<size_t>(in_width)),
                          span_of(scales, blocks * 4), m.span()};
    if (!addressable(spans[0]) || !addressable(spans[2]) || !disjoint(spans, 2, 3)) return RS_ERROR_INVALID_VALUE;
    const rs::QuantizeWeightsWork w{weights, out, scales, weights_stride, weights_expert, experts, out_width, in_width};
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(blocks, kMaxGrid));
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_row(in_width, rs::kVec<T>, [&](auto row) {
            return launch_kernel(RS_KERNEL_QUANTIZE, stream, [&] {
                run_kernel(rs::quantize_weights_kernel<T, decltype(row)::value>, grid, rs::kGateBlock, stream, w);
            });
        });
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_gate_rows(const void *rows, int dtype, size_t num_rows, int width, size_t rows_stride,
                       const int32_t *offsets, int experts, int act, void *out, size_t out_stride, int all,
                       hipStream_t stream) {
    return gate_rows(nullptr, 0, rows, dtype, num_rows, width, rows_stride, offsets, experts, act, out, out_stride, all,
                     false, stream);
}

rs_status rs_gate_rows_backward(const void *grad, size_t grad_stride, const void *rows, int dtype, size_t num_rows,
                                int width, size_t rows_stride, const int32_t *offsets, int experts, int act,
                                void *grad_rows, size_t grad_rows_stride, int all, hipStream_t stream) {
    return gate_rows(grad, grad_stride, rows, dtype, num_rows, width, rows_stride, offsets, experts, act, grad_rows,
                     grad_rows_stride, all, true, stream);
}

rs_status rs_gate_quantize_rows(const void *rows, int dtype, size_t num_rows, int width, size_t rows_stride,
                                const int32_t *offsets, int experts, int act, uint8_t *out, size_t out_stride,
                                float *scales, int all, hipStream_t stream) {
    return quantize_rows(rows, dtype, num_rows, width, rows_stride, offsets, experts, true, act, out, out_stride, scales,
                         all, stream);
}

}  // extern "C"
