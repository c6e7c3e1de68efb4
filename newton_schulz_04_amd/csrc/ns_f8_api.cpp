// ns_f8_api.cpp -- the C ABI of the layers in 8-bit floating point (include/ns.h,
// ns_f8_*): checks the arguments on the host, cuts each product into workgroups by a
// rule on its own sizes, and enqueues the kernels of ns_f8.hip on the caller's stream.
// Descriptors go up as kernel arguments: nothing is allocated, uploaded or kept.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <limits>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_check.h"
#include "ns_enqueue.h"
#include "ns_f8.h"

namespace {

using namespace ns;

// Workgroups of a launch: HIP takes fewer than 2^32 threads at once, 256 a workgroup
// or 512 (products).
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1, kMaxProductGroups = (int64_t(1) << 23) - 1;
constexpr int64_t kMaxLd = std::numeric_limits<int32_t>::max();

int64_t blocks_of(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

ns_status check_kind(int32_t format, int32_t scale_type, int32_t square)
{
    if (format != NS_F8_E4M3 && format != NS_F8_E5M2)
        return fail(NS_EINVAL, "unknown 8-bit format " + std::to_string(format));
    if (scale_type != NS_F8_SCALE_FP32 && scale_type != NS_F8_SCALE_POW2)
        return fail(NS_EINVAL, "unknown scale type " + std::to_string(scale_type));
    if (square != 0 && square != 1)
        return fail(NS_EINVAL, "square must be 0 or 1");
    return NS_OK;
}

ns_status check_dtype(int32_t dtype)
{
    return dtype == NS_BF16 || dtype == NS_FP32 ? NS_OK : fail(NS_EDTYPE, "unknown dtype " + std::to_string(dtype));
}

// q of a matrix, rows of `cols` bytes, and its scales, `per` a block of columns.
ns_status check_q(int32_t i, const char* name, const void* q, int64_t rows, int64_t cols, int64_t ld, int64_t max_ld)
{
    const ns_status st = check_operand(i, name, q, rows, cols, ld, max_ld, 1);
    if (st != NS_OK || rows == 0 || cols == 0)
        return st;
    if (reinterpret_cast<uintptr_t>(q) % 16 || ld % 16)
        return fail(NS_EINVAL, nth(i, name) + " is not aligned to 16 bytes, or its pitch is not a multiple of 16");
    return NS_OK;
}

ns_status check_scale(int32_t i, const char* name, const void* s, int64_t blocks, int64_t per, int64_t ld, int32_t type)
{
    const bool pow2 = type == NS_F8_SCALE_POW2;
    const ns_status st = check_operand(i, name, s, blocks, per, ld, kMaxLd, pow2 ? 1 : 4);
    if (st != NS_OK || blocks == 0 || per == 0)
        return st;
    if (pow2 && (reinterpret_cast<uintptr_t>(s) % 4 || ld % 4))
        return fail(NS_EINVAL, nth(i, name) + " is not aligned to 4 bytes, or its pitch is not a multiple of 4");
    return NS_OK;
}

// The bytes that a quantise call writes for one form of a matrix.
void add_spans(std::vector<Span>& out, int32_t i, const void* q, int64_t rows, int64_t cols, int64_t ld,
               const void* s, int64_t blocks, int64_t per, int64_t ld_s, int32_t type)
{
    const int64_t elt = type == NS_F8_SCALE_POW2 ? 1 : 4;
    out.push_back({reinterpret_cast<uintptr_t>(q), rows, cols, ld, i});
    out.push_back({reinterpret_cast<uintptr_t>(s), blocks, per * elt, ld_s * elt, i});
}

// --- values ------------------------------------------------------------------
ns_status quantize(const ns_f8_rows* mats, int32_t count, int32_t format, int32_t scale_type, int32_t square,
                   int32_t dtype, hipStream_t stream)
{
    ns_status st;
    if (count < 0)
        return fail(NS_EINVAL, "count must be >= 0");
    if ((st = check_kind(format, scale_type, square)) != NS_OK || (st = check_dtype(dtype)) != NS_OK)
        return st;
    if (count > 0 && !mats)
        return fail(NS_EINVAL, "mats must not be NULL when count > 0");
    const int64_t elt = dtype == NS_BF16 ? 2 : 4, selt = scale_type == NS_F8_SCALE_POW2 ? 1 : 4;
    std::vector<Span> spans;
    for (int32_t i = 0; i < count; ++i) {
        const ns_f8_rows& m = mats[i];
        if ((st = check_dim(i, m.rows)) != NS_OK || (st = check_dim(i, m.cols)) != NS_OK)
            return st;
        if (m.rows == 0 || m.cols == 0)
            continue;
        if ((st = check_operand(i, "values", m.values, m.rows, m.cols, m.ld_values, kMaxLd, (size_t)elt)) != NS_OK)
            return st;
        if (!m.q != !m.scale || !m.qt != !m.scale_t)
            return fail(NS_EINVAL, nth(i, "an output's values and scales must both be given, or neither"));
        if (!m.q && !m.qt)
            return fail(NS_EINVAL, nth(i, "no output is given"));
        const int64_t br = blocks_of(m.rows), bc = blocks_of(m.cols);
        const int64_t per = square ? br : m.rows, per_t = square ? bc : m.cols;
        if (m.q) {
            if ((st = check_q(i, "q", m.q, m.rows, m.cols, m.ld_q, kMaxLd)) != NS_OK ||
                (st = check_scale(i, "scale", m.scale, bc, per, m.ld_scale, scale_type)) != NS_OK)
                return st;
            add_spans(spans, i, m.q, m.rows, m.cols, m.ld_q, m.scale, bc, per, m.ld_scale, scale_type);
        }
        if (m.qt) {
            if ((st = check_q(i, "qt", m.qt, m.cols, m.rows, m.ld_qt, kMaxLd)) != NS_OK ||
                (st = check_scale(i, "scale_t", m.scale_t, br, per_t, m.ld_scale_t, scale_type)) != NS_OK)
                return st;
            add_spans(spans, i, m.qt, m.cols, m.rows, m.ld_qt, m.scale_t, br, per_t, m.ld_scale_t, scale_type);
        }
    }
    if ((st = check_spans(spans)) != NS_OK)
        return st;
    F8RowsBatch b;
    b.count = 0;
    b.square = square;
    int64_t nwg = 0;
    auto flush = [&]() -> ns_status {
        if (b.count == 0)
            return NS_OK;
        const hipError_t e =
            launch_f8_quantize(b, (int)nwg, format, scale_type == NS_F8_SCALE_POW2, dtype, stream);
        b.count = 0;
        nwg = 0;
        return launched(e, "8-bit float quantise", stream);
    };
    for (int32_t i = 0; i < count; ++i) {
        const ns_f8_rows& m = mats[i];
        if (m.rows == 0 || m.cols == 0)
            continue;
        // (a matrix of more tiles than a launch takes goes by ranges of whole blocks of
        // rows)
        const int64_t ntn = blocks_of(m.cols);
        for (int64_t row = 0; row < m.rows;) {
            if ((kMaxGroups - nwg) / ntn == 0 && (st = flush()) != NS_OK)
                return st;
            const int64_t some = std::min(m.rows - row, (kMaxGroups - nwg) / ntn * kF8Block), br = row / kF8Block;
            F8RowsItem& it = b.it[b.count++];
            it.values = static_cast<const char*>(m.values) + row * m.ld_values * elt;
            it.q = m.q ? static_cast<char*>(m.q) + row * m.ld_q : nullptr;
            it.scale = m.q ? static_cast<char*>(m.scale) + (square ? br : row) * selt : nullptr;
            it.qt = m.qt ? static_cast<char*>(m.qt) + row : nullptr;
            it.scale_t = m.qt ? static_cast<char*>(m.scale_t) + br * m.ld_scale_t * selt : nullptr;
            it.ldv = m.ld_values;
            it.ldq = m.ld_q;
            it.ldqt = m.ld_qt;
            it.lds = (int32_t)(m.q ? m.ld_scale : 0);
            it.ldst = (int32_t)(m.qt ? m.ld_scale_t : 0);
            it.rows = (int32_t)some;
            it.cols = (int32_t)m.cols;
            it.ntn = (int32_t)ntn;
            it.begin = (int32_t)nwg;
            nwg += blocks_of(some) * ntn;
            row += some;
            if (b.count == kF8RowsItems && (st = flush()) != NS_OK)
                return st;
        }
    }
    return flush();
}

ns_status check_matrix(int32_t i, const char* name, const ns_f8_matrix& m, int64_t max_ld)
{
    ns_status st;
    if ((st = check_kind(m.format, m.scale_type, m.square)) != NS_OK || (st = check_dim(i, m.rows)) != NS_OK ||
        (st = check_dim(i, m.cols)) != NS_OK || (st = check_q(i, name, m.q, m.rows, m.cols, m.ld_q, max_ld)) != NS_OK)
        return st;
    if (m.rows == 0 || m.cols == 0)
        return NS_OK;
    return check_scale(i, "a scale", m.scale, blocks_of(m.cols), m.square ? blocks_of(m.rows) : m.rows, m.ld_scale,
                       m.scale_type);
}

ns_status dequantize(const ns_f8_values* mats, int32_t count, int32_t dtype, hipStream_t stream)
{
    ns_status st;
    if (count < 0)
        return fail(NS_EINVAL, "count must be >= 0");
    if ((st = check_dtype(dtype)) != NS_OK)
        return st;
    if (count > 0 && !mats)
        return fail(NS_EINVAL, "mats must not be NULL when count > 0");
    const int64_t elt = dtype == NS_BF16 ? 2 : 4;
    std::vector<Span> spans;
    for (int32_t i = 0; i < count; ++i) {
        const ns_f8_matrix& m = mats[i].matrix;
        if ((st = check_matrix(i, "q", m, kMaxLd)) != NS_OK ||
            (st = check_operand(i, "values", mats[i].values, m.rows, m.cols, mats[i].ld_values, kMaxLd, (size_t)elt)) !=
                NS_OK)
            return st;
        if (m.rows && m.cols)
            spans.push_back({reinterpret_cast<uintptr_t>(mats[i].values), m.rows, m.cols * elt,
                             mats[i].ld_values * elt, i});
    }
    if ((st = check_spans(spans)) != NS_OK)
        return st;
    F8ValuesBatch b;
    b.count = 0;
    int64_t nwg = 0;
    auto flush = [&]() -> ns_status {
        if (b.count == 0)
            return NS_OK;
        const hipError_t e = launch_f8_dequantize(b, (int)nwg, dtype, stream);
        b.count = 0;
        nwg = 0;
        return launched(e, "8-bit float dequantise", stream);
    };
    for (int32_t i = 0; i < count; ++i) {
        const ns_f8_matrix& m = mats[i].matrix;
        if (m.rows == 0 || m.cols == 0)
            continue;
        // (ranges of 128 rows at least, so that squares stay whole: they take at most
        // 2^21 workgroups)
        const int64_t each = f8_values_wgs(kF8Block, m.cols, elt);
        for (int64_t row = 0; row < m.rows;) {
            if ((kMaxGroups - nwg) / each == 0 && (st = flush()) != NS_OK)
                return st;
            const int64_t some = std::min(m.rows - row, (kMaxGroups - nwg) / each * kF8Block);
            const int64_t selt = m.scale_type == NS_F8_SCALE_POW2 ? 1 : 4;
            F8ValuesItem& it = b.it[b.count++];
            it.q = static_cast<const char*>(m.q) + row * m.ld_q;
            it.scale = static_cast<const char*>(m.scale) + (m.square ? row / kF8Block : row) * selt;
            it.values = static_cast<char*>(mats[i].values) + row * mats[i].ld_values * elt;
            it.ldq = m.ld_q;
            it.ldv = mats[i].ld_values;
            it.lds = (int32_t)m.ld_scale;
            it.rows = (int32_t)some;
            it.cols = (int32_t)m.cols;
            it.kind = m.format | m.scale_type << 1 | m.square << 2;
            it.begin = (int32_t)nwg;
            nwg += f8_values_wgs(some, m.cols, elt);
            row += some;
            if (b.count == kF8ValuesItems && (st = flush()) != NS_OK)
                return st;
        }
    }
    return flush();
}

// --- products ----------------------------------------------------------------
struct Product {
    F8Item item;
    int format;              // of A
    int any;                 // 0: all scales are of one byte; 1; 2: B's are for squares
    size_t part;             // offset of its pieces in the workspace
    enum Kind { kFew16, kFew32, kSmall, kMid, kBig, kNone } kind;
    int64_t groups;
};

// Estimated time of tiles, measured with cold operands: 256 at a time, one a compute unit
// (small ones share it in pairs, which overlaps them but makes them no faster), `block` us
// for each block of k and `each` us beside that. bf16 outputs of one-byte scales, 4096 x
// 8192 of k = 512, 1024, 2048, 4096, 6144: small tiles 28, 43, 71, 135, 216 us, mid 34, 53, 77,
// 126, 204, large 40, 47, 66, 107, 161; fp32 outputs of k = 2048, 6144: 122, 338 small, 129,
// 346 mid, 120, 331 large; fp32 scales, k = 6144: 265 small, 276 mid (a single round of
// small tiles with fp32 scales takes 46 us rather than the 33 of these figures). Mid tiles
// are for bf16 outputs of one-byte scales and fp32 outputs of others (has_mid): for the
// other two they cost more than the two small ones that they hold, however many.
struct Cost { double block, each; };
Cost cost_of(Product::Kind kind, int any, int32_t dtype)
{
    const bool wide = dtype == NS_FP32;
    if (kind == Product::kBig)
        return wide ? Cost{3.3, 7.5} : Cost{1.37, 13};
    if (kind == Product::kMid)
        return wide ? Cost{1.95, 5} : Cost{0.9, 5};
    return any ? (wide ? Cost{1.1, 2} : Cost{0.65, 2}) : wide ? Cost{0.84, 2} : Cost{0.5, 1.5};
}

int64_t tiles_of(Product::Kind kind, const F8Item& it)
{
    const int bm = kind == Product::kBig ? kF8Big : kind == Product::kMid ? kF8MidM : kF8SmallM;
    const int bn = kind == Product::kBig ? kF8Big : kind == Product::kMid ? kF8MidN : kF8SmallN;
    return (int64_t)((it.m + bm - 1) / bm) * ((it.n + bn - 1) / bn);
}

// The products of a list that tiles of a kind are to take, and what they cost.
class Tiled {
public:
    Tiled(Product::Kind kind, int32_t dtype) : kind_(kind), dtype_(dtype) {}
    void add(const Product& p)
    {
        const int64_t n = tiles_of(kind_, p.item), blocks = blocks_of(p.item.k);
        const Cost c = cost_of(kind_, p.any, dtype_);
        tiles_ += n;
        most_ = std::max(most_, blocks);
        block_ += (double)n * blocks * c.block;
        each_ += (double)n * c.each;
        elems_ += (double)p.item.m * p.item.n;
    }
    // us of these products with sums cut in `pieces`, which meet in a second launch: about
    // 5 us, and their own traffic, written and read once at about 6 TB/s (much of it from
    // the last-level cache).
    double us(int pieces = 1) const
    {
        if (tiles_ == 0)
            return 0;
        const double rounds = (double)((tiles_ * pieces + 255) / 256);
        return rounds * (block_ / pieces + each_) / (double)tiles_ + (pieces > 1 ? 5 + pieces * elems_ * 8 / 6e6 : 0);
    }
    // The number of pieces with the least estimated time.
    int pieces() const
    {
        constexpr int64_t kLeast = 2;   // blocks of a piece
        int best = 1;
        for (int p : {2, 3, 4, 6, 8, 10, 12, 14, 16, 20, 24, 28, 32})
            if (most_ >= p * kLeast && us(p) < us(best))
                best = p;
        return best;
    }

private:
    Product::Kind kind_;
    int32_t dtype_;
    int64_t tiles_ = 0, most_ = 0;
    double block_ = 0, each_ = 0, elems_ = 0;
};

// What the large tiles take: one-byte scales, outputs that go four at a time. Sizes alone
// plan a list, so that its cuts, its workspace and its bits depend on nothing else; where an
// output then lies otherwise than in fours, other tiles take the product, its sum in one piece
// (4096 x 8192 by k = 6144 in 184 us instead of 149; 2456 x 3240 by 15540 in 166 instead of
// 142, 159 if the small tiles' sums were cut there).
bool big_by_size(const Product& p) { return !p.any && p.item.n % 4 == 0; }
bool big_by_place(const Product& p, int64_t elt)
{
    return p.item.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(p.item.out) % (4 * elt) == 0;
}

// Checks the products and lays out their work. *bytes: workspace.
ns_status plan(const ns_f8_product* products, int32_t count, int32_t dtype, std::vector<Product>* out, size_t* bytes)
{
    ns_status st;
    if (count < 0)
        return fail(NS_EINVAL, "count must be >= 0");
    if ((st = check_dtype(dtype)) != NS_OK)
        return st;
    if (count > 0 && !products)
        return fail(NS_EINVAL, "products must not be NULL when count > 0");
    const int64_t elt = dtype == NS_BF16 ? 2 : 4;
    std::vector<Span> spans;
    size_t ws = 0;
    int64_t few = 0;   // workgroups of 16 rows of B
    for (int32_t i = 0; i < count; ++i) {
        const ns_f8_matrix &a = products[i].a, &b = products[i].b;
        if ((st = check_matrix(i, "a", a, kMaxPitch)) != NS_OK || (st = check_matrix(i, "b", b, kMaxPitch)) != NS_OK)
            return st;
        if (a.cols != b.cols)
            return fail(NS_EINVAL, nth(i, "a and b have different numbers of columns"));
        if (b.format != NS_F8_E4M3)
            return fail(NS_EINVAL, nth(i, "b must be e4m3"));
        if (a.cols > kMaxPitch)
            return fail(NS_EINVAL, nth(i, "a has more than 2^21 columns"));
        Product p{};
        F8Item& it = p.item;
        it.m = (int32_t)a.rows;
        it.n = (int32_t)b.rows;
        it.k = (int32_t)a.cols;
        if (it.m == 0 || it.n == 0)
            continue;
        if ((st = check_operand(i, "out", products[i].out, it.m, it.n, products[i].ld_out, kMaxPitch, (size_t)elt)) !=
            NS_OK)
            return st;
        spans.push_back({reinterpret_cast<uintptr_t>(products[i].out), it.m, it.n * elt, products[i].ld_out * elt, i});
        it.out = products[i].out;
        it.ldo = (int32_t)products[i].ld_out;
        p.format = a.format;
        if (it.k == 0) {
            // a sum over nothing: the join alone
            p.kind = Product::kNone;
            it.nsplit = 0;
            out->push_back(p);
            continue;
        }
        it.a = static_cast<const char*>(a.q);
        it.b = static_cast<const char*>(b.q);
        it.sa = static_cast<const char*>(a.scale);
        it.sb = static_cast<const char*>(b.scale);
        it.lda = (int32_t)a.ld_q;
        it.ldb = (int32_t)b.ld_q;
        it.ldsa = (int32_t)a.ld_scale;
        it.ldsb = (int32_t)b.ld_scale;
        it.flags = (a.scale_type == NS_F8_SCALE_POW2 ? kF8PowA : 0) | (b.scale_type == NS_F8_SCALE_POW2 ? kF8PowB : 0) |
                   (a.square ? kF8SquareA : 0) | (b.square ? kF8SquareB : 0);
        p.any = (it.flags & (kF8PowA | kF8PowB)) == (kF8PowA | kF8PowB) ? 0 : b.square ? 2 : 1;
        it.nsplit = 1;
        if (it.m <= kF8Few) {
            p.kind = Product::kFew16;
            few += (it.n + 15) / 16;
            out->push_back(p);
            continue;
        }
        p.kind = Product::kSmall;
        if (tiles_of(p.kind, it) > kMaxProductGroups)
            return fail(NS_EINVAL, nth(i, "the output has more than 2^23 - 1 tiles of 128 x 128"));
        out->push_back(p);
    }
    // 16 rows of B a workgroup while that is one for each compute unit at most, else 32, which
    // share a read of A: 16 rows of A, k = 6144, n = 4096: 10.3 us with 16, 11.3 with 32; n = 8192: 15.4
    // and 11.7; 32 rows of A: 11.3 and 14.4; 20.8 and 14.8. (It does not show in the bits.)
    for (Product& p : *out)
        if (p.kind == Product::kFew16) {
            const int rows = few > 256 ? 32 : 16;
            p.kind = few > 256 ? Product::kFew32 : Product::kFew16;
            p.groups = (p.item.n + rows - 1) / rows;
        }
    // Tiles by what they would take of the chip's time: large ones for the products that can
    // have them, mid ones for the others of which there are any, where that is less than with
    // small ones; sums of small tiles are cut where those leave compute units idle. (No kind of
    // tile shows in the bits, a cut does.)
    for (Product::Kind kind : {Product::kBig, Product::kMid}) {
        auto takes = [&](const Product& p) {
            return p.kind == Product::kSmall && (kind == Product::kMid ? has_mid(p.any, dtype) : big_by_size(p));
        };
        Tiled tiled(kind, dtype), mid(Product::kMid, dtype), small(Product::kSmall, dtype);
        for (const Product& p : *out)
            if (takes(p)) {
                tiled.add(p);
                mid.add(p);
                small.add(p);
            }
        double other = small.us(small.pieces());
        if (kind == Product::kBig && has_mid(0, dtype))
            other = std::min(other, mid.us());
        if (tiled.us() < other)
            for (Product& p : *out)
                if (takes(p))
                    p.kind = kind;
    }
    Tiled small(Product::kSmall, dtype);
    for (const Product& p : *out)
        if (p.kind == Product::kSmall)
            small.add(p);
    const int want = small.pieces();
    // (large tiles' products that lie otherwise: uncut, as those would take them)
    Tiled odd_small(Product::kSmall, dtype), odd_mid(Product::kMid, dtype);
    for (Product& p : *out)
        if (p.kind == Product::kBig && !big_by_place(p, elt)) {
            odd_small.add(p);
            odd_mid.add(p);
        }
    const Product::Kind odd = has_mid(0, dtype) && odd_mid.us() < odd_small.us() ? Product::kMid : Product::kSmall;
    for (Product& p : *out) {
        if (p.kind == Product::kFew16 || p.kind == Product::kFew32 || p.kind == Product::kNone)
            continue;
        F8Item& it = p.item;
        const bool big = p.kind == Product::kBig;
        if (big && !big_by_place(p, elt))
            p.kind = odd;
        const int64_t n = tiles_of(p.kind, it), blocks = blocks_of(it.k);
        const int cut = p.kind == Product::kSmall && !big && n * want <= kMaxProductGroups ? want : 1;
        const int bn = p.kind == Product::kBig ? kF8Big : p.kind == Product::kMid ? kF8MidN : kF8SmallN;
        it.ntn = (it.n + bn - 1) / bn;
        it.per = (int32_t)((blocks + cut - 1) / cut);
        it.nsplit = (int32_t)((blocks + it.per - 1) / it.per);
        p.groups = n * it.nsplit;
        if (it.nsplit > 1) {
            p.part = ws;
            ws += ((size_t)it.nsplit * it.m * it.n * 4 + 255) / 256 * 256;
        }
    }
    if ((st = check_spans(spans)) != NS_OK)
        return st;
    *bytes = ws;
    return NS_OK;
}

// Enqueues a planned list: launches of products of one kind and type, then the sums of
// split ones.
class Enqueue {
public:
    Enqueue(float beta, int32_t dtype, char* ws, hipStream_t stream) : dtype_(dtype), ws_(ws), stream_(stream)
    {
        b_.beta = beta;
    }

    ns_status run(std::vector<Product>& work)
    {
        ns_status st = NS_OK;
        for (Product& p : work)
            p.item.part = reinterpret_cast<float*>(ws_ + p.part);
        for (Product::Kind kind : {Product::kFew16, Product::kFew32, Product::kBig, Product::kMid, Product::kSmall})
            for (int format : {0, 1})
                for (int any : {0, 1, 2}) {
                    auto flush = [&]() { return flush_products(kind, format, any); };
                    for (Product& p : work)
                        if (st == NS_OK && p.kind == kind && p.format == format && p.any == any)
                            st = add(p.item, p.groups, kMaxProductGroups, flush);
                    if (st == NS_OK)
                        st = flush();
                }
        auto flush = [&]() { return flush_joins(); };
        for (Product& p : work)
            if (st == NS_OK && p.item.nsplit != 1)
                st = join(p.item, flush);
        return st == NS_OK ? flush() : st;
    }

private:
    template <typename F>
    ns_status add(const F8Item& item, int64_t groups, int64_t most, F&& flush)
    {
        const ns_status st = b_.count == kF8Items || nwg_ + groups > most ? flush() : NS_OK;
        if (st != NS_OK)
            return st;
        F8Item& it = b_.it[b_.count++];
        it = item;
        it.begin = (int32_t)nwg_;
        nwg_ += groups;
        return NS_OK;
    }

    // A sum over nothing may have more outputs than a launch takes: ranges of its rows.
    template <typename F>
    ns_status join(const F8Item& it, F&& flush)
    {
        auto groups = [&](int64_t rows) { return (rows * it.n + kF8JoinElems - 1) / kF8JoinElems; };
        const int64_t step = it.nsplit == 0 ? std::min<int64_t>(it.m, kMaxGroups * kF8JoinElems / it.n) : it.m;
        for (int64_t row = 0; row < it.m; row += step) {
            F8Item part = it;
            part.m = (int32_t)std::min<int64_t>(step, it.m - row);
            part.out = static_cast<char*>(it.out) + row * it.ldo * (dtype_ == NS_BF16 ? 2 : 4);
            const ns_status st = add(part, groups(part.m), kMaxGroups, flush);
            if (st != NS_OK)
                return st;
        }
        return NS_OK;
    }

    ns_status flush_products(Product::Kind kind, int format, int any)
    {
        if (b_.count == 0)
            return NS_OK;
        const hipError_t e = kind == Product::kFew16   ? launch_f8_few(b_, (int)nwg_, 16, format, any, dtype_, stream_)
                             : kind == Product::kFew32 ? launch_f8_few(b_, (int)nwg_, 32, format, any, dtype_, stream_)
                             : kind == Product::kBig ? launch_f8_big(b_, (int)nwg_, format, dtype_, stream_)
                             : kind == Product::kSmall
                                 ? launch_f8_small(b_, (int)nwg_, format, any, dtype_, stream_)
                                                     : launch_f8_mid(b_, (int)nwg_, format, any, dtype_, stream_);
        b_.count = 0;
        nwg_ = 0;
        return launched(e, "8-bit float product", stream_);
    }

    ns_status flush_joins()
    {
        if (b_.count == 0)
            return NS_OK;
        const hipError_t e = launch_f8_join(b_, (int)nwg_, dtype_, stream_);
        b_.count = 0;
        nwg_ = 0;
        return launched(e, "8-bit float product's sum", stream_);
    }

    int32_t dtype_;
    char* ws_;
    hipStream_t stream_;
    F8Batch b_{};
    int64_t nwg_ = 0;
};

}  // namespace

extern "C" {

ns_status ns_f8_quantize(const ns_f8_rows* mats, int32_t count, int32_t format, int32_t scale_type, int32_t square,
                         int32_t dtype, void* stream)
{
    return guarded(
        [&] { return quantize(mats, count, format, scale_type, square, dtype, static_cast<hipStream_t>(stream)); });
}

ns_status ns_f8_dequantize(const ns_f8_values* mats, int32_t count, int32_t dtype, void* stream)
{
    return guarded([&] { return dequantize(mats, count, dtype, static_cast<hipStream_t>(stream)); });
}

ns_status ns_f8_matmul(const ns_f8_product* products, int32_t count, float beta, int32_t dtype, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> ns_status {
        std::vector<Product> work;
        size_t need = 0;
        const ns_status st = plan(products, count, dtype, &work, &need);
        if (st != NS_OK)
            return st;
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(NS_EINVAL,
                        "a workspace of " + std::to_string(need) + " bytes is needed (ns_f8_workspace_bytes)");
        if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 16)
            return fail(NS_EINVAL, "the workspace is not aligned to 16 bytes");
        return Enqueue(beta, dtype, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)).run(work);
    });
}

ns_status ns_f8_workspace_bytes(const ns_f8_product* products, int32_t count, int32_t dtype, size_t* out_bytes)
{
    return guarded([&]() -> ns_status {
        if (!out_bytes)
            return fail(NS_EINVAL, "out_bytes must not be NULL");
        std::vector<Product> work;
        size_t need = 0;
        const ns_status st = plan(products, count, dtype, &work, &need);
        if (st == NS_OK)
            *out_bytes = need;
        return st;
    });
}

}  // extern "C"
