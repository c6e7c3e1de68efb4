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
constexpr int64_t kMaxGroups = int64_t(1) << 30;   // workgroups of one product

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
        b.it[b.count++] = {m.values, m.q, m.scale, m.ld_values, m.ld_q, (int32_t)m.rows, (int32_t)m.cols,
                           (int32_t)nwg};
        nwg += (m.rows + per - 1) / per;
        if (b.count == ns::kQ8RowsItems && (st = flush()) != NS_OK)
            return st;
    }
    return flush();
}

// --- products ----------------------------------------------------------------
struct Product {
    ns::Q8Item item;
    size_t part;     // offset of its pieces in the workspace
    int64_t groups;  // workgroups
    bool big;        // the large tile kernel
};

// How many pieces the k axis of a product is cut into: enough for three
// workgroups on each of the 256 compute units when the output alone has fewer
// tiles, but not below eight slots a piece, where the pieces' own traffic
// (written and read once in 32 bits) would outgrow the operands'.
int pieces(int64_t tiles, int64_t slots)
{
    constexpr int64_t kWant = 768, kMinSlots = 8, kMost = 32;
    if (tiles >= kWant || slots < 2 * kMinSlots)
        return 1;
    return (int)std::max<int64_t>(1, std::min({kWant / tiles, slots / kMinSlots, kMost}));
}

// Whether a product takes the large tiles: they need 16-byte operands, and
// enough outputs to be worth a compute unit each.
bool large(int op, const ns::Q8Item& it)
{
    const int64_t elt = op == NS_Q8_MATMUL ? 1 : 2;
    if ((reinterpret_cast<uintptr_t>(it.a) | reinterpret_cast<uintptr_t>(it.b)) % 16 || it.lda * elt % 16 ||
        it.ldb % 16)
        return false;
    const int64_t tiles = int64_t((it.m + ns::kQ8Big - 1) / ns::kQ8Big) * ((it.n + ns::kQ8Big - 1) / ns::kQ8Big);
    return it.k > 0 && it.m > 128 && it.n > 128 && tiles >= 64;
}

// Checks the layers of a product and lays out its work. *bytes: workspace.
ns_status plan(int op, const ns_q8_layer* layers, int32_t count, int32_t dtype, std::vector<Product>* out,
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
    size_t ws = 0;
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
        } else {
            it.a = l.dy;
            it.lda = (int32_t)l.ld_dy;
            it.b = op == NS_Q8_GRAD_INPUT ? l.wq : l.xq;
            it.ldb = (int32_t)(op == NS_Q8_GRAD_INPUT ? l.ld_wq : l.ld_xq);
            it.sb = op == NS_Q8_GRAD_INPUT ? l.w_scale : l.x_scale;
        }
        it.out = l.out;
        it.ldo = (int32_t)l.ld_out;
        const int64_t slots = (it.k + ns::q8_slot_k(op) - 1) / ns::q8_slot_k(op);
        p.big = large(op, it);
        const int edge = p.big ? ns::kQ8Big : ns::kQ8Tile;
        const int64_t ntm = (it.m + edge - 1) / edge;
        it.ntn = (it.n + edge - 1) / edge;
        const int want = p.big ? 1 : pieces(ntm * it.ntn, slots);
        it.per = (int32_t)std::max<int64_t>(1, (slots + want - 1) / want);
        it.nsplit = (int32_t)std::max<int64_t>(1, (slots + it.per - 1) / it.per);
        p.groups = ntm * it.ntn * it.nsplit;
        if (p.groups > kMaxGroups)
            return fail(NS_EINVAL, nth(i, "the output is too large"));
        if (it.nsplit > 1) {
            p.part = ws;
            ws += ((size_t)it.nsplit * it.m * it.n * 4 + 255) / 256 * 256;
        }
        out->push_back(p);
    }
    if ((st = check_spans(spans)) != NS_OK)
        return st;
    *bytes = ws;
    return NS_OK;
}

ns_status product(int op, const ns_q8_layer* layers, int32_t count, float beta, int32_t dtype, void* workspace,
                  size_t workspace_bytes, hipStream_t stream)
{
    std::vector<Product> work;
    size_t need = 0;
    ns_status st = plan(op, layers, count, dtype, &work, &need);
    if (st != NS_OK)
        return st;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(NS_EINVAL, "a workspace of " + std::to_string(need) + " bytes is needed (ns_q8_workspace_bytes)");
    if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(NS_EINVAL, "the workspace is not aligned to 16 bytes");
    ns::Q8Batch b;
    b.beta = beta;
    // the large tiles, the plain ones, then the sums of the split ones
    for (int pass = 0; pass < 3; ++pass) {
        b.count = 0;
        int64_t nwg = 0;
        auto flush = [&]() -> ns_status {
            if (b.count == 0)
                return NS_OK;
            const hipError_t e = pass == 0   ? ns::launch_q8_big(op, b, (int)nwg, dtype, stream)
                                 : pass == 1 ? ns::launch_q8_tile(op, b, (int)nwg, dtype, stream)
                                             : ns::launch_q8_join(op, b, (int)nwg, dtype, stream);
            b.count = 0;
            nwg = 0;
            return launched(e, pass < 2 ? "8-bit product" : "8-bit product's sum", stream);
        };
        for (Product& p : work) {
            if (pass == 2 ? p.item.nsplit == 1 : p.big != (pass == 0))
                continue;
            const int64_t elems = (int64_t)p.item.m * p.item.n;
            const int64_t groups = pass < 2 ? p.groups : (elems + ns::kQ8JoinElems - 1) / ns::kQ8JoinElems;
            if (b.count == ns::kQ8Items || nwg + groups > kMaxGroups)
                if ((st = flush()) != NS_OK)
                    return st;
            p.item.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part);
            p.item.begin = (int32_t)nwg;
            b.it[b.count++] = p.item;
            nwg += groups;
        }
        if ((st = flush()) != NS_OK)
            return st;
    }
    return NS_OK;
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
        const ns_status st = plan(op, layers, count, dtype, &work, &need);
        if (st == NS_OK)
            *out_bytes = need;
        return st;
    });
}

}  // extern "C"
