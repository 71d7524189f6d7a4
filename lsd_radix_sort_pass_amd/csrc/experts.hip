// experts.hip -- C ABI of the mixture-of-experts calls (routing, slots sorted
// by expert, rows dispatched and combined): argument checks and launches.
// Compiled behind rs.hip (librs.hip), whose helpers it uses.
#include <algorithm>

#include "experts.hpp"

namespace {

constexpr unsigned kMaxGrid = 1u << 20;  // workgroups; the kernels stride over the rest

int dtype_bytes(int dtype) {
    switch (dtype) {
        case RS_F32: return 4;
        case RS_F16:
        case RS_BF16: return 2;
        default: return 0;
    }
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes that `count` rows of `width` elements span.
size_t span_bytes(size_t count, size_t width, size_t stride, size_t elem) {
    return count == 0 ? 0 : ((count - 1) * stride + width) * elem;
}

// A present, aligned array; or any pointer for an empty one.
bool good(const void *p, size_t count, size_t align) { return count == 0 || (p != nullptr && aligned(p, align)); }

constexpr size_t kMaxStride = size_t{1} << 40;

// Whether the rows of an array are addressable and, for an output, disjoint.
bool good_rows(const void *p, size_t count, int width, size_t stride, size_t elem, bool output) {
    if (!good(p, count, elem)) return false;
    if (count <= 1) return true;
    if (stride > kMaxStride || (count - 1) > (size_t{1} << 62) / ((stride + 1) * elem)) return false;
    return !output || stride >= static_cast<size_t>(width);
}

bool disjoint(const Span *spans, int outputs, int all) {
    for (int o = 0; o < outputs; ++o) {
        for (int i = o + 1; i < all; ++i) {
            if (spans[o].lo != spans[o].hi && spans[i].lo != spans[i].hi && overlap(spans[o], spans[i])) return false;
        }
    }
    return true;
}

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
template <int N>
using IntC = std::integral_constant<int, N>;

// Calls f(first row, rows, workgroups) for launches that cover `tokens` rows
// of `lanes` threads each: one, until the threads of a launch reach 2^28.
template <class F>
bool in_parts(size_t tokens, int lanes, F &&f) {
    const size_t per_group = static_cast<size_t>(rs::kRouteBlock / lanes), part = size_t{kMaxGrid} * per_group;
    bool ok = true;
    for (size_t from = 0; ok && from < tokens; from += part) {
        const size_t rows = tokens - from < part ? tokens - from : part;
        ok = f(from, rows, static_cast<unsigned>((rows + per_group - 1) / per_group));
    }
    return ok;
}

// Calls f(IntC<V>) with the values a lane holds of a row that `per_lane` of
// them cover.
template <class F>
bool with_values(int per_lane, F &&f) {
    if (per_lane <= 1) return f(IntC<1>{});
    if (per_lane <= 2) return f(IntC<2>{});
    if (per_lane <= 4) return f(IntC<4>{});
    if (per_lane <= 8) return f(IntC<8>{});
    return f(IntC<16>{});
}

template <class F>
bool with_dtype(int dtype, F &&f) {
    switch (dtype) {
        case RS_F32: return f(float{});
        case RS_F16: return f(rs::f16{});
        default: return f(rs::bf16{});
    }
}

// Whether k choices among rows of `values` logits in each of `lanes` lanes are
// counted rather than taken in rounds, whose time grows as k * (values + 3):
// 2^22 float32 logits, in us, counted / in rounds: 64 experts, k = 4 10.1 / 9.2,
// k = 6 10.4 / 10.9; 128 experts, k = 2 8.1 / 7.1, k = 4 8.1 / 8.4; 1024 experts,
// k = 4 9.8 / 9.5, k = 8 9.8 / 12.4.
bool by_counts(int k, int lanes, int values) { return 2 * k <= lanes && k * (values + 3) > 2 * lanes; }

bool good_route(int dtype, size_t tokens, int experts, int k, int gate) {
    return dtype_bytes(dtype) != 0 && experts >= 1 && experts <= RS_MAX_EXPERTS && k >= 1 && k <= experts &&
           k <= RS_MAX_CHOICES && (gate == RS_GATE_SOFTMAX || gate == RS_GATE_SIGMOID) &&
           tokens <= RS_MAX_SLOTS / static_cast<size_t>(k);
}

// ---------------------------------------------------------------------------
// Slots sorted by expert
// ---------------------------------------------------------------------------
// Up to kOneGroup slots one workgroup places them all: 8192 slots of 256
// experts take it 6.1 us, the two launches below 8.0; for 12000 slots (16 a
// thread) it would take 8.7, as they do.  Above, the slots are cut into at most
// rs::kMaxChunks chunks of whole tiles (one per CU), counted by one launch and
// placed by another, which sums the table of counts itself while that has at
// most kSumWords words, since every workgroup reads it: 2^18 slots of 256
// experts (64 KiB) 9.6 us against 11.9 with a launch that scans it between the
// two, 2^20 slots of 256 experts (256 KiB) 13.4 against 14.5, but of 320 experts
// 15.9 against 14.9 and of 1024 experts 23.3 against 17.2.
constexpr size_t kOneGroup = 8 * rs::kPlaceBlock;
constexpr int kTileItems = 4;
constexpr size_t kTile = size_t{kTileItems} * rs::kPlaceBlock;
constexpr size_t kSumWords = 65536;

struct ExpertPlan {
    size_t chunk = 0;
    unsigned chunks = 1;
};

ExpertPlan expert_plan(size_t n) {
    ExpertPlan p;
    const size_t tiles = (n + kTile - 1) / kTile;
    const size_t per_chunk = (tiles + rs::kMaxChunks - 1) / rs::kMaxChunks;
    p.chunk = (per_chunk ? per_chunk : 1) * kTile;
    p.chunks = static_cast<unsigned>(n ? (n + p.chunk - 1) / p.chunk : 1);
    return p;
}

size_t expert_temp(size_t n, int experts) {
    if (n <= kOneGroup) return 0;
    // The table, and a row of totals.
    const size_t bytes = (size_t{expert_plan(n).chunks} + 1) * rs::table_stride(static_cast<uint32_t>(experts)) * 4;
    return align_up(bytes);
}

bool good_experts(size_t n, int experts) {
    return experts >= 1 && experts <= RS_MAX_EXPERTS && n <= RS_MAX_SLOTS;
}

template <class ID>
rs_status sort_experts(const ID *ids, size_t n, int first, int experts, int32_t *order, int32_t *position,
                       int32_t *offsets, void *temp, size_t temp_bytes, hipStream_t stream) {
    if (!good_experts(n, experts) || first < 0 || first > INT32_MAX - experts + 1) return RS_ERROR_INVALID_VALUE;
    if (!good(ids, n, sizeof(ID)) || !good(order, n, 4) || !good(position, n, 4) || !good(offsets, 1, 4)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const size_t need = expert_temp(n, experts);
    if (need != 0) {
        if (!temp || !aligned(temp, kTempAlign)) return RS_ERROR_INVALID_VALUE;
        if (temp_bytes < need) return RS_ERROR_INSUFFICIENT_TEMP;
    }
    const Span spans[] = {span_of(order, n * 4), span_of(position, n * 4),
                          span_of(offsets, 4 * (static_cast<size_t>(experts) + 1)), span_of(temp, need),
                          span_of(ids, n * sizeof(ID))};
    if (!disjoint(spans, 4, 5)) return RS_ERROR_INVALID_VALUE;

    const auto e = static_cast<uint32_t>(experts);
    const auto f = static_cast<ID>(first);
    auto *table = static_cast<uint32_t *>(temp);
    const ExpertPlan p = expert_plan(n);
    uint32_t *totals = table + size_t{p.chunks} * rs::table_stride(e);
    const auto place = [&](auto kernel, unsigned grid, size_t chunk) {
        return launch_kernel(RS_KERNEL_EXPERT, stream, [&] {
            run_kernel(kernel, grid, rs::kPlaceBlock, stream, ids, n, f, e, chunk, table, totals, g_ranker == 1, order,
                       position, offsets);
        });
    };
    const auto run = [&](auto keys) {
        constexpr int kKeys = decltype(keys)::value;
        if (n <= rs::kPlaceBlock) return place(rs::expert_place_kernel<ID, 1, kKeys, rs::kNoTable>, 1, n);
        if (n <= 4 * rs::kPlaceBlock) return place(rs::expert_place_kernel<ID, 4, kKeys, rs::kNoTable>, 1, n);
        if (n <= kOneGroup) return place(rs::expert_place_kernel<ID, 8, kKeys, rs::kNoTable>, 1, n);
        bool ok = launch_kernel(RS_KERNEL_EXPERT, stream, [&] {
            run_kernel(rs::expert_count_kernel<ID, kTileItems>, p.chunks, rs::kPlaceBlock, stream, ids, n, f, e, p.chunk,
                       table);
        });
        if (p.chunks * size_t{rs::table_stride(e)} <= kSumWords) {
            return ok && place(rs::expert_place_kernel<ID, kTileItems, kKeys, rs::kCounts>, p.chunks, p.chunk);
        }
        ok = ok && launch_kernel(RS_KERNEL_EXPERT, stream, [&] {
            const unsigned grid = grid_for(rs::table_stride(e), 4 * rs::kScanQuads, kMaxGrid);
            run_kernel(rs::expert_scan_kernel, grid, rs::kPlaceBlock, stream, table, p.chunks, e, totals);
        });
        return ok && place(rs::expert_place_kernel<ID, kTileItems, kKeys, rs::kScanned>, p.chunks, p.chunk);
    };
    const bool ok = experts <= 256 ? run(std::integral_constant<int, 256>{}) : run(std::integral_constant<int, 1024>{});
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
bool good_shape(int dtype, size_t tokens, int width, int k, size_t num_rows) {
    return dtype_bytes(dtype) != 0 && width >= 1 && width <= RS_MAX_ROW_WIDTH && k >= 1 && k <= RS_MAX_CHOICES &&
           tokens <= RS_MAX_SLOTS / static_cast<size_t>(k) && num_rows <= RS_MAX_SLOTS;
}

// Calls f(integral_constant B) with the batch for k slots: the fewest batches
// of at most kMaxBatch, of even size.
template <class F>
bool with_batch(int k, F &&f) {
    const int batches = (k + rs::kMaxBatch - 1) / rs::kMaxBatch;
    const int size = (k + batches - 1) / batches;
    if (size <= 1) return f(std::integral_constant<int, 1>{});
    if (size <= 2) return f(std::integral_constant<int, 2>{});
    if (size <= 4) return f(std::integral_constant<int, 4>{});
    if (size <= 6) return f(std::integral_constant<int, 6>{});
    return f(std::integral_constant<int, 8>{});
}

// The one batch of a join with dots.
template <class F>
bool with_whole_batch(int k, F &&f) {
    if (k <= rs::kMaxBatch) return with_batch(k, f);
    if (k <= 10) return f(std::integral_constant<int, 10>{});
    if (k <= 12) return f(std::integral_constant<int, 12>{});
    return f(std::integral_constant<int, rs::kMaxJoinBatch>{});
}

// Calls f(IntC<U>) with the chunks that are in flight together in batches of B
// slots: at most 8 accesses, evenly over the rounds, since a lane behind the
// row's end still reads.  float32 rows of 4096, two slots: 65.1 us for 4093
// tokens, 69.1 one by one.
template <int B, class F>
bool with_at_once(int chunks, F &&f) {
    constexpr int kMost = B <= 2 ? 4 : B <= 4 ? 2 : 1;
    const int rounds = (chunks + kMost - 1) / kMost, at_once = (chunks + rounds - 1) / rounds;
    if constexpr (kMost >= 4) {
        if (at_once == 4) return f(IntC<4>{});
        if (at_once == 3) return f(IntC<3>{});
    }
    if constexpr (kMost >= 2) {
        if (at_once == 2) return f(IntC<2>{});
    }
    return f(IntC<1>{});
}

constexpr size_t kLastLevelBytes = size_t{1} << 28;  // the memory-side cache of an MI355X

// Enqueues the spread or the join of w, with its dots if w.dots is set.
template <bool SPREAD, class T>
bool launch_rows(rs::RowWork<T> w, hipStream_t stream) {
    const int vecs = (w.width + rs::kVec<T> - 1) / rs::kVec<T>;
    const size_t clearing = w.clear_rows ? (w.num_rows + w.clear_rows - 1) / w.clear_rows : 0;  // workgroups
    const auto go = [&](auto kernel, size_t units, int per_block) {
        w.clearing = static_cast<unsigned>(clearing);
        const unsigned grid = w.clearing + grid_for(units, static_cast<unsigned>(per_block), kMaxGrid);
        return launch_kernel(RS_KERNEL_ROWS, stream, [&] { run_kernel(kernel, grid, rs::kRowBlock, stream, w); });
    };
    const bool weighted = w.weights != nullptr;
    if (vecs <= rs::kNarrow) {
        w.lanes = 1;
        while (w.lanes < vecs) w.lanes *= 2;
        const int per_block = rs::kRowBlock / w.lanes;
        const auto narrow = [&](auto dots) {
            constexpr bool kDots = decltype(dots)::value;
            return weighted ? go(rs::narrow_rows_kernel<T, SPREAD, true, kDots>, w.tokens, per_block)
                            : go(rs::narrow_rows_kernel<T, SPREAD, false, kDots>, w.tokens, per_block);
        };
        return w.dots ? narrow(std::true_type{}) : narrow(std::false_type{});
    }
    const size_t arrays = w.tokens + w.num_rows * (SPREAD && w.dots != nullptr ? 2 : 1);  // rows in all
    w.once = arrays * static_cast<size_t>(w.width) >= kLastLevelBytes / sizeof(T);
    if (w.dots != nullptr && (SPREAD || w.k <= rs::kMaxJoinBatch)) {
        const auto whole = [&](auto batch) {
            constexpr int B = decltype(batch)::value;
            if (vecs <= 64) {
                w.chunks = 1;
                return weighted ? go(rs::wide_rows_kernel<T, 64, B, 1, SPREAD, true, true, false>, w.tokens, rs::kRowBlock / 64)
                                : go(rs::wide_rows_kernel<T, 64, B, 1, SPREAD, false, true, false>, w.tokens, rs::kRowBlock / 64);
            }
            constexpr int L = rs::kRowBlock;
            w.chunks = (vecs + L - 1) / L;
            return with_at_once<B>(w.chunks, [&](auto at_once) {
                constexpr int U = decltype(at_once)::value;
                return weighted ? go(rs::wide_rows_kernel<T, L, B, U, SPREAD, true, true, false>, w.tokens, 1)
                                : go(rs::wide_rows_kernel<T, L, B, U, SPREAD, false, true, false>, w.tokens, 1);
            });
        };
        return SPREAD ? with_batch(w.k, whole) : with_whole_batch(w.k, whole);
    }
    constexpr int kWaves = rs::kRowBlock / 64;
    constexpr size_t kMaxGridY = 65535;
    w.chunks = (vecs + 63) / 64;
    w.side = w.chunks >= 3 ? 2 : w.chunks - 1;
    static_assert(kWaves == 4);
    const size_t per_block = kWaves >> w.side, blocks = (w.tokens + per_block - 1) / per_block;
    const auto across = static_cast<unsigned>((w.chunks + (1 << w.side) - 1) >> w.side);
    w.clearing = static_cast<unsigned>((clearing + across - 1) / across);
    const size_t most = kMaxGridY - w.clearing;
    const dim3 grid(across, w.clearing + static_cast<unsigned>(blocks < most ? blocks : most));
    const auto plain = [&](auto batch) {
        constexpr int B = decltype(batch)::value;
        const auto run = [&](auto kernel) {
            return launch_kernel(RS_KERNEL_ROWS, stream, [&] { run_kernel(kernel, grid, rs::kRowBlock, stream, w); });
        };
        if constexpr (!SPREAD) {
            if (w.once) {
                return weighted ? run(rs::wide_rows_kernel<T, 64, B, 1, false, true, false, true>)
                                : run(rs::wide_rows_kernel<T, 64, B, 1, false, false, false, true>);
            }
        }
        return weighted ? run(rs::wide_rows_kernel<T, 64, B, 1, SPREAD, true, false, false>)
                        : run(rs::wide_rows_kernel<T, 64, B, 1, SPREAD, false, false, false>);
    };
    // A spread without dots loads no rows: its batch only unrolls the stores.
    const bool ok = SPREAD ? plain(std::integral_constant<int, rs::kMaxBatch>{}) : with_batch(w.k, plain);
    const size_t slots = w.tokens * static_cast<size_t>(w.k);
    return ok && (w.dots == nullptr || go(rs::dot_rows_kernel<T>, slots, rs::kRowBlock / 64));
}

// Whether the rows that no slot names are cleared by kClearGroups groups of the
// spread's own launch, which read all places each while the spread takes its
// time, or all rows are by a launch before.  Not at all / beside / before, in us,
// bfloat16, k = 8, with dots: 2048 x 128 9.1 / 9.1 / 11.3, 8192 x 128 12.7 / 14.0 /
// 17.6, 32768 x 128 32 / 51 / 44, 32768 x 256 59 / 65 / 78, 8192 x 2048 91 / 91 / 126;
// without: 3000 x 128 6.5 / 6.5 / 8.8, 8192 x 128 7 / 13 / 11, 32768 x 256 25 / 49 /
// 44, 32768 x 512 51 / 69 / 87, 32768 x 1024 106 / 108 / 181; with dots for 1000 rows
// of 512 among 500000 x 8 slots 349 / 614 / 369.  More slots than 2^22 would not fit
// the groups' bits.
constexpr size_t kClearGroups = 64;
bool clear_beside(size_t slots, size_t num_rows, size_t row_bytes, bool dots) {
    if (num_rows > slots || slots > kClearGroups * rs::kClearRows) return false;
    const size_t hides = (dots ? 512 : 1024) / (slots <= (size_t{1} << 16) ? 4 : 1);  // bytes of rows a slot
    return slots <= (size_t{1} << 14) || num_rows * row_bytes >= slots * hides;
}

// Enqueues zeros in whole rows.
bool launch_clear(int dtype, void *rows, size_t num_rows, int width, size_t stride, hipStream_t stream) {
    return with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        const int vecs = (width + rs::kVec<T> - 1) / rs::kVec<T>;
        int lanes = 1;
        while (lanes < vecs && lanes < rs::kRowBlock) lanes *= 2;
        const unsigned grid = grid_for(num_rows, static_cast<unsigned>(rs::kRowBlock / lanes), kMaxGrid);
        return launch_kernel(RS_KERNEL_ROWS, stream, [&] {
            run_kernel(rs::clear_rows_kernel<T>, grid, rs::kRowBlock, stream, static_cast<T *>(rows), num_rows, width,
                       stride, lanes);
        });
    });
}

// all: rows that no slot names are cleared.
bool launch_spread(int dtype, const void *x, size_t tokens, int width, size_t x_stride, const int32_t *position,
                   const float *weights, int k, void *rows, size_t num_rows, size_t rows_stride, const void *rows_in,
                   size_t rows_in_stride, float *dots, bool all, hipStream_t stream) {
    const size_t row_bytes = static_cast<size_t>(width) * static_cast<size_t>(dtype_bytes(dtype));
    const bool clear = all && num_rows != 0;
    const bool beside = clear && clear_beside(tokens * static_cast<size_t>(k), num_rows, row_bytes, dots != nullptr);
    if (clear && !beside && !launch_clear(dtype, rows, num_rows, width, rows_stride, stream)) return false;
    if (tokens == 0 || (num_rows == 0 && dots == nullptr)) return true;
    return with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        rs::RowWork<T> w{};
        w.x = static_cast<const T *>(x), w.x_stride = x_stride;
        w.rows_in = static_cast<const T *>(rows_in), w.rows_in_stride = rows_in_stride;
        w.rows_out = static_cast<T *>(rows), w.rows_out_stride = rows_stride;
        w.dots = dots, w.position = position, w.weights = weights;
        w.tokens = tokens, w.num_rows = num_rows, w.width = width, w.k = k;
        if (beside) {
            const size_t groups = std::min(kClearGroups, (num_rows + 255) / 256);
            w.clear_rows = static_cast<uint32_t>((num_rows + 32 * groups - 1) / (32 * groups) * 32);
        }
        return launch_rows<true>(w, stream);
    });
}

bool launch_join(int dtype, const void *rows, size_t num_rows, size_t rows_stride, const int32_t *position,
                 const float *weights, int k, void *out, size_t tokens, int width, size_t out_stride, const void *x,
                 size_t x_stride, float *dots, hipStream_t stream) {
    if (tokens == 0) return true;
    return with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        rs::RowWork<T> w{};
        w.x = static_cast<const T *>(x), w.x_stride = x_stride;
        w.rows_in = static_cast<const T *>(rows), w.rows_in_stride = rows_stride;
        w.out = static_cast<T *>(out), w.out_stride = out_stride;
        w.dots = dots, w.position = position, w.weights = weights;
        w.tokens = tokens, w.num_rows = num_rows, w.width = width, w.k = k;
        return launch_rows<false>(w, stream);
    });
}

rs_status combine_backward(const void *grad_out, int dtype, size_t tokens, int width, size_t grad_out_stride,
                           const int32_t *position, const float *weights, int k, const void *rows, size_t rows_stride,
                           void *grad_rows, size_t grad_rows_stride, size_t num_rows, float *grad_weights, bool all,
                           hipStream_t stream) {
    if (!good_shape(dtype, tokens, width, k, num_rows)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), slots = tokens * static_cast<size_t>(k);
    if (!good_rows(grad_out, tokens, width, grad_out_stride, elem, false) || !good(position, slots, 4) ||
        !good_rows(grad_rows, num_rows, width, grad_rows_stride, elem, true) || (weights && !aligned(weights, 4))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const bool dots = grad_weights != nullptr;
    if (dots && (!aligned(grad_weights, 4) || !good_rows(rows, num_rows, width, rows_stride, elem, false))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const auto w = static_cast<size_t>(width);
    const Span spans[] = {span_of(grad_rows, span_bytes(num_rows, w, grad_rows_stride, elem)),
                          span_of(grad_weights, dots ? slots * 4 : 0),
                          span_of(grad_out, span_bytes(tokens, w, grad_out_stride, elem)),
                          span_of(position, slots * 4), span_of(weights, weights ? slots * 4 : 0),
                          span_of(rows, dots ? span_bytes(num_rows, w, rows_stride, elem) : 0)};
    if (!disjoint(spans, 2, 6)) return RS_ERROR_INVALID_VALUE;
    const bool ok = launch_spread(dtype, grad_out, tokens, width, grad_out_stride, position, weights, k, grad_rows,
                                  num_rows, grad_rows_stride, rows, rows_stride, grad_weights, all, stream);
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

}  // namespace

extern "C" {

rs_status rs_route_topk(const void *logits, int dtype, size_t tokens, int experts, size_t stride, int k, int gate,
                        int renormalize, float scale, float *weights_out, int32_t *experts_out, hipStream_t stream) {
    if (!good_route(dtype, tokens, experts, k, gate)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), slots = tokens * static_cast<size_t>(k);
    if (!good_rows(logits, tokens, experts, stride, elem, false) || !good(weights_out, slots, 4) ||
        !good(experts_out, slots, 4)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const Span spans[] = {span_of(weights_out, slots * 4), span_of(experts_out, slots * 4),
                          span_of(logits, span_bytes(tokens, static_cast<size_t>(experts), stride, elem))};
    if (!disjoint(spans, 2, 3)) return RS_ERROR_INVALID_VALUE;
    if (tokens == 0) return RS_SUCCESS;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        const auto go = [&](auto kernel, int lanes, bool counts) {
            return in_parts(tokens, lanes, [&](size_t from, size_t rows, unsigned grid) {
                return launch_kernel(RS_KERNEL_ROUTE, stream, [&] {
                    run_kernel(kernel, grid, rs::kRouteBlock, stream, static_cast<const T *>(logits) + from * stride,
                               rows, experts, stride, k, gate, renormalize, scale, counts, weights_out + from * k,
                               experts_out + from * k);
                });
            });
        };
        // At most 16 logits a lane, and two lanes a choice.
        const auto with_lanes = [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            return with_values((experts + kLanes - 1) / kLanes, [&](auto v) {
                constexpr int kValues = decltype(v)::value;
                return go(rs::route_topk_kernel<T, kLanes, kValues>, kLanes, by_counts(k, kLanes, kValues));
            });
        };
        if (k <= 8 && experts <= 256) return with_lanes(IntC<16>{});
        if (k <= 16 && experts <= 512) return with_lanes(IntC<32>{});
        return with_lanes(IntC<64>{});
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_route_topk_backward(const void *logits, int dtype, size_t tokens, int experts, size_t stride,
                                 const int32_t *chosen, const float *grad_weights, int k, int gate, int renormalize,
                                 float scale, void *grad_logits, size_t grad_stride, hipStream_t stream) {
    if (!good_route(dtype, tokens, experts, k, gate)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), slots = tokens * static_cast<size_t>(k);
    if (!good_rows(logits, tokens, experts, stride, elem, false) || !good(chosen, slots, 4) ||
        !good(grad_weights, slots, 4) || !good_rows(grad_logits, tokens, experts, grad_stride, elem, true)) {
        return RS_ERROR_INVALID_VALUE;
    }
    const auto row = static_cast<size_t>(experts);
    const Span spans[] = {span_of(grad_logits, span_bytes(tokens, row, grad_stride, elem)), span_of(chosen, slots * 4),
                          span_of(grad_weights, slots * 4), span_of(logits, span_bytes(tokens, row, stride, elem))};
    if (!disjoint(spans, 1, 4)) return RS_ERROR_INVALID_VALUE;
    if (tokens == 0) return RS_SUCCESS;
    const bool ok = with_dtype(dtype, [&](auto zero) {
        using T = decltype(zero);
        const auto go = [&](auto kernel, int lanes) {
            return in_parts(tokens, lanes, [&](size_t from, size_t rows, unsigned grid) {
                return launch_kernel(RS_KERNEL_ROUTE, stream, [&] {
                    run_kernel(kernel, grid, rs::kRouteBlock, stream, static_cast<const T *>(logits) + from * stride,
                               rows, experts, stride, chosen + from * k, grad_weights + from * k, k, gate, renormalize,
                               scale, static_cast<T *>(grad_logits) + from * grad_stride, grad_stride);
                });
            });
        };
        const int by16 = (experts + 15) / 16, by64 = (experts + 63) / 64;
        if (k <= 16 && by16 <= 16) {
            return with_values(by16, [&](auto v) {
                return go(rs::route_topk_backward_kernel<T, 16, decltype(v)::value>, 16);
            });
        }
        return with_values(by64, [&](auto v) {
            return go(rs::route_topk_backward_kernel<T, 64, decltype(v)::value>, 64);
        });
    });
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

size_t rs_temp_bytes_experts(size_t n, int experts) { return good_experts(n, experts) ? expert_temp(n, experts) : 0; }

rs_status rs_sort_experts_i32(const int32_t *ids, size_t n, int first, int experts, int32_t *order_out,
                              int32_t *position_out, int32_t *offsets_out, void *temp, size_t temp_bytes,
                              hipStream_t stream) {
    return sort_experts(ids, n, first, experts, order_out, position_out, offsets_out, temp, temp_bytes, stream);
}

rs_status rs_sort_experts_i64(const int64_t *ids, size_t n, int first, int experts, int32_t *order_out,
                              int32_t *position_out, int32_t *offsets_out, void *temp, size_t temp_bytes,
                              hipStream_t stream) {
    return sort_experts(ids, n, first, experts, order_out, position_out, offsets_out, temp, temp_bytes, stream);
}

rs_status rs_dispatch_rows(const void *x, int dtype, size_t tokens, int width, size_t x_stride,
                           const int32_t *position, const float *weights, int k, void *rows, size_t num_rows,
                           size_t rows_stride, hipStream_t stream) {
    if (!good_shape(dtype, tokens, width, k, num_rows)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), slots = tokens * static_cast<size_t>(k);
    if (!good_rows(x, tokens, width, x_stride, elem, false) || !good(position, slots, 4) ||
        !good_rows(rows, num_rows, width, rows_stride, elem, true) || (weights && !aligned(weights, 4))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const auto w = static_cast<size_t>(width);
    const Span spans[] = {span_of(rows, span_bytes(num_rows, w, rows_stride, elem)),
                          span_of(x, span_bytes(tokens, w, x_stride, elem)), span_of(position, slots * 4),
                          span_of(weights, weights ? slots * 4 : 0)};
    if (!disjoint(spans, 1, 4)) return RS_ERROR_INVALID_VALUE;
    const bool ok = launch_spread(dtype, x, tokens, width, x_stride, position, weights, k, rows, num_rows, rows_stride,
                                  nullptr, 0, nullptr, false, stream);
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_dispatch_rows_backward(const void *grad_rows, int dtype, size_t num_rows, size_t grad_rows_stride,
                                    const int32_t *position, const float *weights, int k, const void *x,
                                    size_t x_stride, void *grad_x, size_t grad_x_stride, float *grad_weights,
                                    size_t tokens, int width, hipStream_t stream) {
    if (!good_shape(dtype, tokens, width, k, num_rows)) return RS_ERROR_INVALID_VALUE;
    const size_t elem = static_cast<size_t>(dtype_bytes(dtype)), slots = tokens * static_cast<size_t>(k);
    if (!good_rows(grad_rows, num_rows, width, grad_rows_stride, elem, false) || !good(position, slots, 4) ||
        !good_rows(grad_x, tokens, width, grad_x_stride, elem, true) || (weights && !aligned(weights, 4))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const bool dots = grad_weights != nullptr;
    if (dots && (!aligned(grad_weights, 4) || !good_rows(x, tokens, width, x_stride, elem, false))) {
        return RS_ERROR_INVALID_VALUE;
    }
    const auto w = static_cast<size_t>(width);
    const Span spans[] = {span_of(grad_x, span_bytes(tokens, w, grad_x_stride, elem)),
                          span_of(grad_weights, dots ? slots * 4 : 0),
                          span_of(grad_rows, span_bytes(num_rows, w, grad_rows_stride, elem)),
                          span_of(position, slots * 4), span_of(weights, weights ? slots * 4 : 0),
                          span_of(x, dots ? span_bytes(tokens, w, x_stride, elem) : 0)};
    if (!disjoint(spans, 2, 6)) return RS_ERROR_INVALID_VALUE;
    const bool ok = launch_join(dtype, grad_rows, num_rows, grad_rows_stride, position, weights, k, grad_x, tokens,
                                width, grad_x_stride, x, x_stride, grad_weights, stream);
    return ok ? RS_SUCCESS : RS_ERROR_LAUNCH;
}

rs_status rs_combine_rows(const void *rows, int dtype, size_t num_rows, size_t rows_stride, const int32_t *position,
                          const float *weights, int k, void *out, size_t tokens, int width, size_t out_stride,
                          hipStream_t stream) {
    return rs_dispatch_rows_backward(rows, dtype, num_rows, rows_stride, position, weights, k, nullptr, 0, out,
                                     out_stride, nullptr, tokens, width, stream);
}

rs_status rs_combine_rows_backward(const void *grad_out, int dtype, size_t tokens, int width, size_t grad_out_stride,
                                   const int32_t *position, const float *weights, int k, const void *rows,
                                   size_t rows_stride, void *grad_rows, size_t grad_rows_stride, size_t num_rows,
                                   float *grad_weights, hipStream_t stream) {
    return combine_backward(grad_out, dtype, tokens, width, grad_out_stride, position, weights, k, rows, rows_stride,
                            grad_rows, grad_rows_stride, num_rows, grad_weights, false, stream);
}

rs_status rs_combine_rows_backward_all(const void *grad_out, int dtype, size_t tokens, int width, size_t grad_out_stride,
                                       const int32_t *position, const float *weights, int k, const void *rows,
                                       size_t rows_stride, void *grad_rows, size_t grad_rows_stride, size_t num_rows,
                                       float *grad_weights, hipStream_t stream) {
    return combine_backward(grad_out, dtype, tokens, width, grad_out_stride, position, weights, k, rows, rows_stride,
                            grad_rows, grad_rows_stride, num_rows, grad_weights, true, stream);
}

}  // extern "C"
