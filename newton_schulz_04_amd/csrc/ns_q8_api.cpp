// ns_q8_api.cpp -- the C ABI of the 8-bit linear layers (include/ns.h,
// ns_q8_*): checks the arguments on the host, cuts each product into
// workgroups by a rule on its own sizes, and enqueues the kernels of
// ns_q8.hip on the caller's stream. Descriptors go up as kernel arguments:
// nothing is allocated, uploaded or kept.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <limits>
#include <new>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_enqueue.h"
#include "ns_q8.h"

namespace {

using ns::fail;
using ns::hip_fail;

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxPitch = int64_t(1) << 21;    // of the products' operands
// Workgroups of a launch: HIP takes fewer than 2^32 threads at once, 256 a
// workgroup, or 512 (k_q8_few). What has more goes in several launches, single
// matrices by ranges of rows.
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1, kMaxFewGroups = (int64_t(1) << 23) - 1;

std::string nth(int32_t i, const char* what) { return "matrix " + std::to_string(i) + ": " + what; }

// NS_CHECK=1: wait for the stream after every launch (see ns.h).
ns_status launched(hipError_t e, const char* what, hipStream_t stream)
{
    if (e != hipSuccess)
        return hip_fail(e, what);
    const char* v = std::getenv("NS_CHECK");
    if (v && v[0] == '1' && v[1] == 0) {
        e = hipStreamSynchronize(stream);
        if (e == hipSuccess)
            e = hipGetLastError();
        if (e != hipSuccess)
            return fail(NS_EHIP, std::string("NS_CHECK: the ") + what + " kernel failed (" + hipGetErrorString(e) + ")");
    }
    return NS_OK;
}

// --- outputs -----------------------------------------------------------------
// An output: rows of `len` bytes at a pitch of `pitch` bytes.
struct Span {
    uintptr_t at;
    int64_t rows, len, pitch;
    int32_t index;
    uintptr_t end() const { return at + (uintptr_t)((rows - 1) * pitch + len); }
};

// Two outputs whose byte ranges meet may still be column slices of one wide
// matrix: the same pitch, and columns that do not meet.
bool meet(const Span& a, const Span& b)
{
    if (a.at >= b.end() || b.at >= a.end())
        return false;
    if (a.rows == 1 && b.rows == 1)
        return true;
    const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
    if ((a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) || a.len > pitch || b.len > pitch)
        return true;
    const Span& lo = a.at <= b.at ? a : b;
    const Span& hi = a.at <= b.at ? b : a;
    const int64_t d = (int64_t)((hi.at - lo.at) % (uintptr_t)pitch);   // hi's column in lo's rows
    return !(d >= lo.len && d + hi.len <= pitch);
}

ns_status check_spans(std::vector<Span>& s)
{
    std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
    for (size_t i = 0; i < s.size(); ++i)
        for (size_t j = i + 1; j < s.size() && s[j].at < s[i].end(); ++j)
            if (meet(s[i], s[j]))
                return fail(NS_EINVAL, "the outputs of matrices " + std::to_string(std::min(s[i].index, s[j].index)) +
                                           " and " + std::to_string(std::max(s[i].index, s[j].index)) + " overlap");
    return NS_OK;
}

// A rows x cols operand that the call reads or writes.
ns_status check_operand(int32_t i, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld,
                        int64_t max_ld, size_t elt)
{
    if (rows == 0 || cols == 0)
        return NS_OK;
    if (!p)
        return fail(NS_EINVAL, nth(i, name) + " is non-empty but its pointer is NULL");
    if (reinterpret_cast<uintptr_t>(p) % elt)
        return fail(NS_EINVAL, nth(i, name) + " is not aligned to its element size");
    if (ld < cols)
        return fail(NS_EINVAL, nth(i, name) + " has a pitch below its row length");
    if (ld > max_ld)
        return fail(NS_EINVAL, nth(i, name) + " has a pitch above " + std::to_string(max_ld));
    return NS_OK;
}

ns_status check_dim(int32_t i, int64_t v)
{
    if (v < 0)
        return fail(NS_EINVAL, nth(i, "a dimension is negative"));
    if (v > kMaxDim)
        return fail(NS_EINVAL, nth(i, "a dimension is above 2^24"));
    return NS_OK;
}

// --- rows --------------------------------------------------------------------
ns_status rows_call(const ns_q8_rows* mats, int32_t count, int32_t mode, int32_t dtype, hipStream_t stream,
                    bool quantize)
{
    if (count < 0)
        return fail(NS_EINVAL, "count must be >= 0");
    if (mode != NS_Q8_ABSMAX && mode != NS_Q8_POW2)
        return fail(NS_EINVAL, "unknown scale mode " + std::to_string(mode));
    if (dtype != NS_BF16 && dtype != NS_FP32)
        return fail(NS_EDTYPE, "unknown dtype " + std::to_string(dtype));
    if (count > 0 && !mats)
        return fail(NS_EINVAL, "mats must not be NULL when count > 0");
    const size_t elt = dtype == NS_BF16 ? 2 : 4;
    std::vector<Span> out;
    ns_status st;
    for (int32_t i = 0; i < count; ++i) {
        const ns_q8_rows& m = mats[i];
        if ((st = check_dim(i, m.rows)) != NS_OK || (st = check_dim(i, m.cols)) != NS_OK)
            return st;
        if (m.rows == 0 || m.cols == 0)
            continue;
        const int64_t max_ld = std::numeric_limits<int32_t>::max();
        if ((st = check_operand(i, "values", m.values, m.rows, m.cols, m.ld_values, max_ld, elt)) != NS_OK ||
            (st = check_operand(i, "q", m.q, m.rows, m.cols, m.ld_q, max_ld, 1)) != NS_OK ||
            (st = check_operand(i, "scale", m.scale, m.rows, 1, 1, 1, 4)) != NS_OK)
            return st;
        if (quantize) {
            out.push_back({reinterpret_cast<uintptr_t>(m.q), m.rows, m.cols, m.ld_q, i});
            out.push_back({reinterpret_cast<uintptr_t>(m.scale), 1, 4 * m.rows, 4 * m.rows, i});
        } else {
            out.push_back({reinterpret_cast<uintptr_t>(m.values), m.rows, m.cols * (int64_t)elt,
                           m.ld_values * (int64_t)elt, i});
        }
    }
    if ((st = check_spans(out)) != NS_OK)
        return st;
    ns::Q8RowsBatch b;
    b.mode = mode;
    b.count = 0;
    int64_t nwg = 0;
    auto flush = [&]() -> ns_status {
        if (b.count == 0)
            return NS_OK;
        const hipError_t e = quantize ? ns::launch_q8_quantize(b, (int)nwg, dtype, stream)
                                      : ns::launch_q8_dequantize(b, (int)nwg, dtype, stream);
        b.count = 0;
        nwg = 0;
        return launched(e, quantize ? "quantise" : "dequantise", stream);
    };
    for (int32_t i = 0; i < count; ++i) {
        const ns_q8_rows& m = mats[i];
        // a matrix without columns has scales all the same, but nothing that
        // they would scale: they are left as they are
        if (m.rows == 0 || m.cols == 0)
            continue;
        const int per = ns::q8_rows_per_wg(m.cols);
        for (int64_t row = 0; row < m.rows;) {
            const int64_t rows = std::min(m.rows - row, (kMaxGroups - nwg) * per);
            b.it[b.count++] = {static_cast<char*>(m.values) + row * m.ld_values * (int64_t)elt,
                               m.q + row * m.ld_q, m.scale + row, m.ld_values, m.ld_q, (int32_t)rows,
                               (int32_t)m.cols, (int32_t)nwg};
            nwg += (rows + per - 1) / per;
            row += rows;
            if ((b.count == ns::kQ8RowsItems || nwg == kMaxGroups) && (st = flush()) != NS_OK)
                return st;
        }
    }
    return flush();
}

// --- products ----------------------------------------------------------------
struct Product {
    ns::Q8Item item;
    size_t part;             // offset of its pieces in the workspace
    int64_t rows_a, rows_b;  // rows and bytes a row of the operands
    int64_t len_a, len_b;
    size_t copy_a, copy_b;   // offsets of their aligned copies, or kNone
    enum Kind { kFew, kBig, kMid, kThin, kNone } kind;
    int64_t groups;          // workgroups (kBig: tiles)
};
constexpr size_t kNone = ~size_t(0);

int64_t tiles_of(const ns::Q8Item& it, int edge)
{
    return (int64_t)((it.m + edge - 1) / edge) * ((it.n + edge - 1) / edge);
}

// How many pieces the k axis of `tiles` tiles of 128 x 128 and `slots` slots is
// cut into: the number with the least estimated time. Measured on tiles of
// grad_weight and matmul: 0.3 us a slot and round of tiles over the 256 compute
// units; sums split over pieces pay a second launch, about 4 us, and
// their own traffic, written and read once at about 4 TB/s (2048 x 2048 outputs of
// k = 1024 take 17 us whole and 38 us in two pieces; 18 x 2304 of k = 8192 about
// 80 us whole and 12 us in 14 pieces).
int pieces(int64_t tiles, int64_t slots, double elems, int64_t at_once = 256, double us_slot = 0.3)
{
    constexpr int64_t kLeast = 4;   // slots of a piece: fewer leave no pipeline
    int best = 1;
    double least = 1e300;
    for (int p : {1, 2, 3, 4, 6, 8, 10, 12, 14, 16, 20, 24, 28, 32}) {
        if (p > 1 && slots < p * kLeast)
            break;
        const double rounds = (double)((tiles * p + at_once - 1) / at_once);
        const double us = rounds * ((slots + p - 1) / p) * us_slot + (p > 1 ? 4 + p * elems * 8 / 4e6 : 0);
        if (us < least) {
            least = us;
            best = p;
        }
    }
    return best;
}

// Whether a product gains from 256 x 256 tiles, given a list that has enough
// of them to fill the compute units: its sums are long enough for one
// workgroup a compute unit to hide its loads and stores behind them, which takes
// longer where a gradient is added to what is there (`adds`), and the tiles'
// edges waste little. Large against small tiles, 4096 x 6144 outputs: matmul 24 us in
// either at k = 512, 34 against 40 us at k = 1024; grad_weight, bf16, 47 against
// 49 us at k = 768, 76 against 85 us at 1536; adding, 56 against 51 us at k = 768,
// 85 against 88 us at 1536, 146 against 161 us at 3000.
bool suits_big(int op, bool adds, const ns::Q8Item& it, int64_t slots)
{
    const int64_t least = op == NS_Q8_MATMUL ? 12 : op == NS_Q8_GRAD_INPUT ? 16 : adds ? 48 : 24;
    return slots >= least && (double)it.m * it.n >= 0.85 * 65536 * tiles_of(it, ns::kQ8Big);
}
// Large tiles that a list needs at least: 192 of them (2048 x 6144) are faster
// than the 768 small ones by a fifth, 64 (2048 x 2048) slower by two thirds.
constexpr int64_t kBigTiles = 160;

// Checks the layers of a product and lays out its work. adds: beta != 0.
// *bytes: workspace, which does not depend on it.
ns_status plan(int op, const ns_q8_layer* layers, int32_t count, bool adds, int32_t dtype, std::vector<Product>* out,
               size_t* bytes)
{
    if (count < 0)
        return fail(NS_EINVAL, "count must be >= 0");
    if (op != NS_Q8_MATMUL && op != NS_Q8_GRAD_INPUT && op != NS_Q8_GRAD_WEIGHT)
        return fail(NS_EINVAL, "unknown product " + std::to_string(op));
    if ((dtype != NS_BF16 && dtype != NS_FP32) || (op == NS_Q8_GRAD_INPUT && dtype != NS_BF16))
        return fail(NS_EDTYPE, op == NS_Q8_GRAD_INPUT && dtype == NS_FP32 ? "the input's gradient is bf16"
                                                                           : "unknown dtype " + std::to_string(dtype));
    if (count > 0 && !layers)
        return fail(NS_EINVAL, "layers must not be NULL when count > 0");
    const size_t elt = dtype == NS_BF16 ? 2 : 4;
    std::vector<Span> spans;
    ns_status st;
    for (int32_t i = 0; i < count; ++i) {
        const ns_q8_layer& l = layers[i];
        const int64_t t = l.tokens, o = l.out_features, k = l.in_features;
        if ((st = check_dim(i, t)) != NS_OK || (st = check_dim(i, o)) != NS_OK || (st = check_dim(i, k)) != NS_OK)
            return st;
        if (op == NS_Q8_MATMUL && k > NS_Q8_MAX_K)
            return fail(NS_EINVAL, nth(i, "in_features is above NS_Q8_MAX_K"));
        Product p{};
        ns::Q8Item& it = p.item;
        it.m = (int32_t)(op == NS_Q8_GRAD_WEIGHT ? o : t);
        it.n = (int32_t)(op == NS_Q8_MATMUL ? o : k);
        it.k = (int32_t)(op == NS_Q8_MATMUL ? k : op == NS_Q8_GRAD_INPUT ? o : t);
        if (it.m == 0 || it.n == 0)
            continue;
        if (op != NS_Q8_GRAD_WEIGHT &&
            ((st = check_operand(i, "wq", l.wq, o, k, l.ld_wq, kMaxPitch, 1)) != NS_OK ||
             (st = check_operand(i, "w_scale", l.w_scale, o, 1, 1, 1, 4)) != NS_OK))
            return st;
        if (op != NS_Q8_GRAD_INPUT &&
            ((st = check_operand(i, "xq", l.xq, t, k, l.ld_xq, kMaxPitch, 1)) != NS_OK ||
             (st = check_operand(i, "x_scale", l.x_scale, t, 1, 1, 1, 4)) != NS_OK))
            return st;
        if (op != NS_Q8_MATMUL && (st = check_operand(i, "dy", l.dy, t, o, l.ld_dy, kMaxPitch, 2)) != NS_OK)
            return st;
        if ((st = check_operand(i, "out", l.out, it.m, it.n, l.ld_out, kMaxPitch, elt)) != NS_OK)
            return st;
        spans.push_back({reinterpret_cast<uintptr_t>(l.out), it.m, it.n * (int64_t)elt, l.ld_out * (int64_t)elt, i});
        if (op == NS_Q8_MATMUL) {
            it.a = l.xq;
            it.lda = (int32_t)l.ld_xq;
            it.b = l.wq;
            it.ldb = (int32_t)l.ld_wq;
            it.sa = l.x_scale;
            it.sb = l.w_scale;
            p.rows_a = t, p.len_a = k;
            p.rows_b = o, p.len_b = k;
        } else {
            it.a = l.dy;
            it.lda = (int32_t)l.ld_dy;
            it.b = op == NS_Q8_GRAD_INPUT ? l.wq : l.xq;
            it.ldb = (int32_t)(op == NS_Q8_GRAD_INPUT ? l.ld_wq : l.ld_xq);
            it.sb = op == NS_Q8_GRAD_INPUT ? l.w_scale : l.x_scale;
            p.rows_a = t, p.len_a = 2 * o;
            p.rows_b = op == NS_Q8_GRAD_INPUT ? o : t, p.len_b = k;
        }
        it.out = l.out;
        it.ldo = (int32_t)l.ld_out;
        if (tiles_of(it, ns::kQ8Mid) > kMaxGroups)
            return fail(NS_EINVAL, nth(i, "the output has more than 2^24 - 1 tiles of 128 x 128"));
        out->push_back(p);
    }
    if ((st = check_spans(spans)) != NS_OK)
        return st;

    size_t ws = 0;
    auto take = [&](size_t n) {
        const size_t at = ws;
        ws += (n + 255) / 256 * 256;
        return at;
    };
    // Integer sums do not depend on how they are cut, so matmul looks at the
    // whole list; the gradients' cut goes by the product's own sizes, so that a
    // layer's bits do not depend on what it shares a call with. (Which tiles
    // a product takes does not show in its bits.)
    int64_t tiles = 0, most_slots = 0, big = 0;
    double elems = 0;
    auto slots_of = [&](const ns::Q8Item& it) {
        return (int64_t)(it.k + ns::q8_slot_k(op) - 1) / ns::q8_slot_k(op);
    };
    for (Product& p : *out) {
        const ns::Q8Item& it = p.item;
        // (k_q8_thin reads 16 bytes from inside a row: a row's worth of either
        // operand has to follow)
        const bool thin = op == NS_Q8_GRAD_WEIGHT && it.m <= ns::kQ8Thin && it.k > 0 && it.lda >= 8 && it.ldb >= 16;
        p.kind = op == NS_Q8_MATMUL && it.m <= ns::kQ8Few ? Product::kFew : thin ? Product::kThin : Product::kMid;
        if (p.kind != Product::kMid || it.k == 0)
            continue;
        tiles += tiles_of(it, ns::kQ8Mid);
        elems += (double)it.m * it.n;
        most_slots = std::max(most_slots, slots_of(it));
        if (suits_big(op, adds, it, slots_of(it)))
            big += tiles_of(it, ns::kQ8Big);
    }
    auto cut = [](ns::Q8Item& it, int64_t slots, int want) {
        it.per = (int32_t)std::max<int64_t>(1, (slots + want - 1) / want);
        it.nsplit = (int32_t)std::max<int64_t>(1, (slots + it.per - 1) / it.per);
    };
    const int list_pieces = op == NS_Q8_MATMUL ? pieces(tiles, most_slots, elems) : 0;
    for (Product& p : *out) {
        ns::Q8Item& it = p.item;
        const int64_t ea = op == NS_Q8_MATMUL ? 1 : 2, slots = slots_of(it);
        p.copy_a = p.copy_b = kNone;
        if (p.kind == Product::kFew) {
            it.nsplit = 1;
            p.groups = (it.n + ns::q8_few_channels(it.m) - 1) / ns::q8_few_channels(it.m);
            continue;
        }
        if (it.k == 0 && tiles == 0) {
            // a sum over nothing, in a list without tiles: the join alone
            p.kind = Product::kNone;
            it.nsplit = 0;
            continue;
        }
        if (p.kind == Product::kThin) {
            it.ntn = (it.n + ns::kQ8Mid - 1) / ns::kQ8Mid;
            cut(it, slots, pieces(it.ntn, slots, (double)it.m * it.n, 384, 0.5));
            p.groups = (int64_t)it.ntn * it.nsplit;
            if (it.nsplit > 1)
                p.part = take((size_t)it.nsplit * it.m * it.n * 4);
            continue;
        }
        auto aligned = [](const void* q, int64_t pitch) {
            return reinterpret_cast<uintptr_t>(q) % 16 == 0 && pitch % 16 == 0;
        };
        if (it.k > 0 && !aligned(it.a, it.lda * ea))
            p.copy_a = take(p.rows_a * ((p.len_a + 15) / 16 * 16));
        if (it.k > 0 && !aligned(it.b, it.ldb))
            p.copy_b = take(p.rows_b * ((p.len_b + 15) / 16 * 16));
        const int want = op == NS_Q8_MATMUL
                             ? list_pieces
                             : pieces(tiles_of(it, ns::kQ8Mid), slots, (double)it.m * it.n);
        cut(it, slots, tiles_of(it, ns::kQ8Mid) * want <= kMaxGroups ? want : 1);
        if (it.nsplit == 1 && big >= kBigTiles && suits_big(op, adds, it, slots))
            p.kind = Product::kBig;
        const int edge = p.kind == Product::kBig ? ns::kQ8Big : ns::kQ8Mid;
        it.ntn = (it.n + edge - 1) / edge;
        p.groups = tiles_of(it, edge) * it.nsplit;
        if (it.nsplit > 1)
            p.part = take((size_t)it.nsplit * it.m * it.n * 4);
    }
    *bytes = ws;
    return NS_OK;
}

// Enqueues the kernels of one product: aligned copies, products of few tokens,
// large and small tiles, products of few rows, sums of split products.
class Enqueue {
public:
    Enqueue(int op, float beta, int32_t dtype, char* ws, hipStream_t stream)
        : op_(op), dtype_(dtype), ws_(ws), stream_(stream)
    {
        b_.beta = beta;
    }

    ns_status run(std::vector<Product>& work)
    {
        ns_status st = copies(work);
        for (Pass pass : {kFew, kBig, kMid, kThin, kJoin}) {
            b_.count = 0;
            nwg_ = 0;
            for (Product& p : work) {
                if (st != NS_OK)
                    return st;
                if (pass == kJoin ? p.item.nsplit == 1 : (int)p.kind != (int)pass)
                    continue;
                p.item.part = reinterpret_cast<float*>(ws_ + p.part);
                st = pass == kJoin ? join(p.item) : add(pass, p.item, p.groups);
            }
            if (st == NS_OK)
                st = flush(pass);
        }
        return st;
    }

private:
    enum Pass {
        kFew = Product::kFew,
        kBig = Product::kBig,
        kMid = Product::kMid,
        kThin = Product::kThin,
        kJoin = Product::kNone + 1   // of sums in several pieces, or none
    };

    ns_status add(Pass pass, ns::Q8Item& it, int64_t groups)
    {
        // (large tiles: room for the halves of the last round)
        const int64_t most = pass == kFew ? kMaxFewGroups : pass == kBig ? kMaxGroups - 128 : kMaxGroups;
        const ns_status st = b_.count == ns::kQ8Items || nwg_ + groups > most ? flush(pass) : NS_OK;
        if (st != NS_OK)
            return st;
        it.begin = (int32_t)nwg_;
        b_.it[b_.count++] = it;
        nwg_ += groups;
        return NS_OK;
    }

    // The pieces of a sum over k added up. A sum over nothing may have more
    // outputs than a launch takes: ranges of its rows.
    ns_status join(const ns::Q8Item& it)
    {
        auto groups = [&](int64_t rows) { return (rows * it.n + ns::kQ8JoinElems - 1) / ns::kQ8JoinElems; };
        const int64_t step = it.nsplit == 0 ? std::min<int64_t>(it.m, kMaxGroups * ns::kQ8JoinElems / it.n) : it.m;
        for (int64_t row = 0; row < it.m; row += step) {
            ns::Q8Item part = it;
            part.m = (int32_t)std::min<int64_t>(step, it.m - row);
            part.out = static_cast<char*>(it.out) + row * it.ldo * (dtype_ == NS_BF16 ? 2 : 4);
            if (it.sa)
                part.sa += row;
            const ns_status st = add(kJoin, part, groups(part.m));
            if (st != NS_OK)
                return st;
        }
        return NS_OK;
    }

    ns_status flush(Pass pass)
    {
        if (b_.count == 0)
            return NS_OK;
        hipError_t e;
        const char* what = "8-bit product";
        if (pass == kFew) {
            e = ns::launch_q8_few(b_, (int)nwg_, dtype_, stream_);
        } else if (pass == kBig) {
            // The last round's tiles, when they would leave at least half of
            // the 256 compute units idle, run as halves on all of them.
            const int64_t last = nwg_ % 256, split = nwg_ > 256 && last <= 128 ? last : 0;
            e = ns::launch_q8_big(op_, b_, (int)(nwg_ + split), (int)(nwg_ - split), dtype_, stream_);
        } else if (pass == kMid) {
            e = ns::launch_q8_mid(op_, b_, (int)nwg_, dtype_, stream_);
        } else if (pass == kThin) {
            e = ns::launch_q8_thin(b_, (int)nwg_, dtype_, stream_);
        } else {
            e = ns::launch_q8_join(op_, b_, (int)nwg_, dtype_, stream_);
            what = "8-bit product's sum";
        }
        b_.count = 0;
        nwg_ = 0;
        return launched(e, what, stream_);
    }

    ns_status copies(std::vector<Product>& work)
    {
        ns::Q8AlignBatch b;
        b.count = 0;
        int64_t nwg = 0;
        auto flush = [&]() -> ns_status {
            if (b.count == 0)
                return NS_OK;
            const hipError_t e = ns::launch_q8_align(b, (int)nwg, stream_);
            b.count = 0;
            nwg = 0;
            return launched(e, "8-bit operand copy", stream_);
        };
        auto add = [&](const void* src, int64_t pitch, int64_t rows, int64_t len, size_t at) -> ns_status {
            const int64_t chunks = (len + 15) / 16, step = kMaxGroups * ns::kQ8AlignChunks / chunks;
            for (int64_t row = 0; row < rows; row += step) {
                const int64_t some = std::min(step, rows - row);
                const int64_t groups = (some * chunks + ns::kQ8AlignChunks - 1) / ns::kQ8AlignChunks;
                if (b.count == ns::kQ8AlignItems || nwg + groups > kMaxGroups) {
                    const ns_status st = flush();
                    if (st != NS_OK)
                        return st;
                }
                b.it[b.count++] = {static_cast<const char*>(src) + row * pitch, ws_ + at + row * chunks * 16, pitch,
                                   (int32_t)some, (int32_t)len, (int32_t)nwg};
                nwg += groups;
            }
            return NS_OK;
        };
        ns_status st = NS_OK;
        const int ea = op_ == NS_Q8_MATMUL ? 1 : 2;
        for (Product& p : work) {
            ns::Q8Item& it = p.item;
            if (st == NS_OK && p.copy_a != kNone) {
                st = add(it.a, (int64_t)it.lda * ea, p.rows_a, p.len_a, p.copy_a);
                it.a = ws_ + p.copy_a;
                it.lda = (int32_t)((p.len_a + 15) / 16 * 16 / ea);
            }
            if (st == NS_OK && p.copy_b != kNone) {
                st = add(it.b, it.ldb, p.rows_b, p.len_b, p.copy_b);
                it.b = reinterpret_cast<const int8_t*>(ws_ + p.copy_b);
                it.ldb = (int32_t)((p.len_b + 15) / 16 * 16);
            }
        }
        return st == NS_OK ? flush() : st;
    }

    int op_;
    int32_t dtype_;
    char* ws_;
    hipStream_t stream_;
    ns::Q8Batch b_{};
    int64_t nwg_ = 0;
};

ns_status product(int op, const ns_q8_layer* layers, int32_t count, float beta, int32_t dtype, void* workspace,
                  size_t workspace_bytes, hipStream_t stream)
{
    std::vector<Product> work;
    size_t need = 0;
    ns_status st = plan(op, layers, count, beta != 0.f, dtype, &work, &need);
    if (st != NS_OK)
        return st;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(NS_EINVAL, "a workspace of " + std::to_string(need) + " bytes is needed (ns_q8_workspace_bytes)");
    if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(NS_EINVAL, "the workspace is not aligned to 16 bytes");
    return Enqueue(op, beta, dtype, static_cast<char*>(workspace), stream).run(work);
}

// Runs an entry point's body: host allocations that fail are NS_ENOMEM.
template <typename F>
ns_status guarded(F&& f)
{
    ns::clear_error();
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return fail(NS_ENOMEM, "host allocation failed");
    }
}

}  // namespace

extern "C" {

ns_status ns_q8_quantize(const ns_q8_rows* mats, int32_t count, int32_t mode, int32_t dtype, void* stream)
{
    return guarded([&] { return rows_call(mats, count, mode, dtype, static_cast<hipStream_t>(stream), true); });
}

ns_status ns_q8_dequantize(const ns_q8_rows* mats, int32_t count, int32_t dtype, void* stream)
{
    return guarded(
        [&] { return rows_call(mats, count, NS_Q8_ABSMAX, dtype, static_cast<hipStream_t>(stream), false); });
}

ns_status ns_q8_matmul(const ns_q8_layer* layers, int32_t count, int32_t dtype, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    return guarded([&] {
        return product(NS_Q8_MATMUL, layers, count, 0.f, dtype, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
    });
}

ns_status ns_q8_grad_input(const ns_q8_layer* layers, int32_t count, void* workspace, size_t workspace_bytes,
                           void* stream)
{
    return guarded([&] {
        return product(NS_Q8_GRAD_INPUT, layers, count, 0.f, NS_BF16, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
    });
}

ns_status ns_q8_grad_weight(const ns_q8_layer* layers, int32_t count, float beta, int32_t dtype, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    return guarded([&] {
        return product(NS_Q8_GRAD_WEIGHT, layers, count, beta, dtype, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
    });
}

ns_status ns_q8_workspace_bytes(int32_t op, const ns_q8_layer* layers, int32_t count, int32_t dtype,
                                size_t* out_bytes)
{
    return guarded([&]() -> ns_status {
        if (!out_bytes)
            return fail(NS_EINVAL, "out_bytes must not be NULL");
        std::vector<Product> work;
        size_t need = 0;
        const ns_status st = plan(op, layers, count, false, dtype, &work, &need);
        if (st == NS_OK)
            *out_bytes = need;
        return st;
    });
}

}  // extern "C"
