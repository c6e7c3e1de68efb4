// The host code of the 8-bit linear layers under AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_q8_sanitizers.py builds this with g++
// and ns_q8_api.cpp). The kernel launchers below only look at what they are
// given: random lists of layers, and for every launch
//   - each item's workgroups follow the previous item's, and cover its output;
//   - the k slots of a split product are covered once by its pieces;
//   - operands are 16-byte aligned for the tile kernels, in place or as a copy
//     that a copy launch made before, with the pitch that the copy has;
//   - copies and pieces lie inside the workspace, apart from one another;
//   - the buffer resources that the tile kernels build over the operands end
//     with them (rounded up to 16 bytes), also where no k is left.
// Prints "q8_check ok" and returns 0 when everything holds.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_enqueue.h"
#include "ns_q8.h"

static int g_fail = 0;
#define EXPECT(cond, ...)                                             \
    do {                                                              \
        if (!(cond)) {                                                \
            std::fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__); \
            std::fprintf(stderr, __VA_ARGS__);                        \
            std::fprintf(stderr, "\n");                               \
            if (++g_fail > 20)                                        \
                std::exit(1);                                         \
        }                                                             \
    } while (0)

namespace ns {
static std::string g_msg;
ns_status fail(ns_status s, const std::string& msg)
{
    g_msg = msg;
    return s;
}
ns_status hip_fail(hipError_t, const char* what) { return fail(NS_EHIP, what); }
void clear_error() { g_msg.clear(); }
}  // namespace ns

namespace {

struct Extent { uintptr_t base; int64_t rows, len, pitch; };   // bytes
std::map<uintptr_t, Extent> g_operands;   // by address: the call's, then copies
std::vector<std::pair<uintptr_t, uintptr_t>> g_taken;   // of the workspace
uintptr_t g_ws, g_ws_end;
std::map<uintptr_t, int> g_written;   // outputs, by address
std::map<uintptr_t, int> g_split;     // of them, still to be joined

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

void take(uintptr_t at, int64_t n)
{
    EXPECT(at >= g_ws && at + n <= g_ws_end, "outside the workspace");
    for (auto& p : g_taken)
        EXPECT(at >= p.second || at + n <= p.first, "workspace used twice");
    g_taken.push_back({at, at + n});
}

const Extent& operand(const void* p)
{
    auto it = g_operands.find(reinterpret_cast<uintptr_t>(p));
    EXPECT(it != g_operands.end(), "an operand that is none");
    return it->second;
}

// bytes [base + at, + n) lie in the operand, rounded up to 16
void inside(const Extent& e, int64_t at, int64_t n)
{
    if (n <= 0)
        return;
    const int64_t end = e.rows && e.len ? up16((e.rows - 1) * e.pitch + e.len) : 0;
    EXPECT(at >= 0 && at + n <= end, "a resource of %lld at %lld passes the operand's %lld", (long long)n,
           (long long)at, (long long)end);
}

// The resources of a tile of bm x bn over slots [s0, s1), with the slots that
// the pipeline asks for past the end.
void tile_resources(int op, const ns::Q8Item& it, int bm, int bn, int64_t m0, int64_t n0, int s0, int s1)
{
    const int slot = ns::q8_slot_k(op), elt = op == ns::kQ8Matmul ? 1 : 2;
    const int64_t rows = std::min<int64_t>(bm, it.m - m0), cols = std::min<int64_t>(bn, it.n - n0);
    const int64_t lda = (int64_t)it.lda * elt, ldb = it.ldb;
    auto krows = [&](int64_t left, int64_t pitch, int64_t width) {
        return left > 0 ? (std::min<int64_t>(slot, left) - 1) * pitch + up16(width) : 0;
    };
    if (it.k == 0)
        return;   // nothing is left at once: no resource is larger than 0 (or read)
    const Extent &a = operand(it.a), &b = operand(it.b);
    EXPECT(a.pitch == lda && b.pitch == ldb, "a pitch that is not the operand's");
    EXPECT((a.base | b.base | lda | ldb) % 16 == 0, "an unaligned operand");
    for (int s : {s0, s0 + 1, (s0 + s1) / 2, s1 - 1, s1, s1 + 4}) {
        const int64_t left = s < s1 ? it.k - (int64_t)s * slot : 0;
        if (op == ns::kQ8GradWeight)
            inside(a, m0 * 2 + (int64_t)s * slot * lda, krows(left, lda, rows * 2));
        if (op != ns::kQ8Matmul)
            inside(b, n0 + (int64_t)s * slot * ldb, krows(left, ldb, cols));
    }
    if (op != ns::kQ8GradWeight)
        inside(a, m0 * lda, up16((rows - 1) * lda + it.k * elt));
    if (op == ns::kQ8Matmul)
        inside(b, n0 * ldb, up16((cols - 1) * ldb + it.k));
}

int64_t tiles_of(const ns::Q8Item& it, int edge)
{
    return (int64_t)((it.m + edge - 1) / edge) * ((it.n + edge - 1) / edge);
}

void tile_launch(int op, const ns::Q8Batch& b, int64_t total, int edge)
{
    EXPECT(b.count > 0 && b.count <= ns::kQ8Items, "items");
    int64_t at = 0;
    for (int i = 0; i < b.count; ++i) {
        const ns::Q8Item& it = b.it[i];
        const int ns_ = (it.k + ns::q8_slot_k(op) - 1) / ns::q8_slot_k(op);
        EXPECT(it.begin == at, "begin");
        EXPECT(it.ntn == (it.n + edge - 1) / edge, "ntn");
        EXPECT(it.nsplit >= 1 && (edge == ns::kQ8Mid || it.nsplit == 1), "nsplit");
        EXPECT((int64_t)it.nsplit * it.per >= ns_ && (int64_t)(it.nsplit - 1) * it.per < std::max(1, ns_),
               "pieces cover the slots, none empty");
        at += tiles_of(it, edge) * it.nsplit;
        for (int64_t m0 = 0; m0 < it.m; m0 += edge)
            for (int64_t n0 = 0; n0 < it.n; n0 += edge)
                if ((m0 == 0 || m0 + edge >= it.m) && (n0 == 0 || n0 + edge >= it.n))
                    for (int p : {0, it.nsplit - 1}) {
                        tile_resources(op, it, edge, edge, m0, n0, p * it.per, std::min(ns_, (p + 1) * it.per));
                        if (edge == ns::kQ8Big)
                            for (int64_t h : {0, 128})
                                if (n0 + h < it.n)
                                    tile_resources(op, it, edge, 128, m0, n0 + h, 0, ns_);
                    }
        const uintptr_t out = reinterpret_cast<uintptr_t>(it.out);
        EXPECT(g_written[out]++ == 0, "an output written twice");
        if (it.nsplit > 1) {
            take(reinterpret_cast<uintptr_t>(it.part), (int64_t)it.nsplit * it.m * it.n * 4);
            g_split[out] = it.nsplit;
        }
    }
    EXPECT(at == total, "workgroups");
}

}  // namespace

namespace ns {
hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int, hipStream_t)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= kQ8RowsItems, "items");
    for (int i = 0; i < b.count; ++i) {
        EXPECT(b.it[i].begin == at, "begin");
        const int per = q8_rows_per_wg(b.it[i].cols);
        at += (b.it[i].rows + per - 1) / per;
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int dt, hipStream_t s)
{
    return launch_q8_quantize(b, nwg, dt, s);
}
hipError_t launch_q8_big(int op, const Q8Batch& b, int nwg, int nwhole, int, hipStream_t)
{
    EXPECT(nwhole > 0 && (nwg - nwhole) % 2 == 0, "halves come in twos");
    tile_launch(op, b, nwhole + (nwg - nwhole) / 2, kQ8Big);
    return hipSuccess;
}
hipError_t launch_q8_mid(int op, const Q8Batch& b, int nwg, int, hipStream_t)
{
    tile_launch(op, b, nwg, kQ8Mid);
    return hipSuccess;
}
hipError_t launch_q8_thin(const Q8Batch& b, int nwg, int, hipStream_t)
{
    int64_t at = 0;
    for (int i = 0; i < b.count; ++i) {
        const Q8Item& it = b.it[i];
        const int ns_ = (it.k + q8_slot_k(kQ8GradWeight) - 1) / q8_slot_k(kQ8GradWeight);
        EXPECT(it.begin == at && it.m <= kQ8Thin && it.k > 0 && it.ntn == (it.n + kQ8Mid - 1) / kQ8Mid, "few rows");
        EXPECT((int64_t)it.nsplit * it.per >= ns_ && (int64_t)(it.nsplit - 1) * it.per < ns_, "pieces");
        at += (int64_t)it.ntn * it.nsplit;
        const uintptr_t out = reinterpret_cast<uintptr_t>(it.out);
        EXPECT(g_written[out]++ == 0, "an output written twice");
        if (it.nsplit > 1) {
            take(reinterpret_cast<uintptr_t>(it.part), (int64_t)it.nsplit * it.m * it.n * 4);
            g_split[out] = it.nsplit;
        }
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_q8_few(const Q8Batch& b, int nwg, int, hipStream_t)
{
    int64_t at = 0;
    for (int i = 0; i < b.count; ++i) {
        const Q8Item& it = b.it[i];
        EXPECT(it.begin == at && it.m <= kQ8Few && it.nsplit == 1, "few tokens");
        at += (it.n + q8_few_channels(it.m) - 1) / q8_few_channels(it.m);
        EXPECT(g_written[reinterpret_cast<uintptr_t>(it.out)]++ == 0, "an output written twice");
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_q8_join(int, const Q8Batch& b, int nwg, int, hipStream_t)
{
    int64_t at = 0;
    for (int i = 0; i < b.count; ++i) {
        const Q8Item& it = b.it[i];
        EXPECT(it.begin == at, "begin");
        at += ((int64_t)it.m * it.n + kQ8JoinElems - 1) / kQ8JoinElems;
        if (it.nsplit == 0) {
            // a sum over nothing
            EXPECT(it.k == 0 && g_written[reinterpret_cast<uintptr_t>(it.out)]++ == 0, "an output written twice");
            continue;
        }
        auto s = g_split.find(reinterpret_cast<uintptr_t>(it.out));
        EXPECT(s != g_split.end() && s->second == it.nsplit, "joins what was split");
        g_split.erase(s);
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_q8_align(const Q8AlignBatch& b, int nwg, hipStream_t)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= kQ8AlignItems, "items");
    for (int i = 0; i < b.count; ++i) {
        const Q8AlignItem& it = b.it[i];
        const Extent e = operand(it.src);
        EXPECT(it.begin == at && it.pitch == e.pitch && it.rows == e.rows && it.len == e.len, "copy");
        at += (it.rows * (up16(it.len) / 16) + kQ8AlignChunks - 1) / kQ8AlignChunks;
        take(reinterpret_cast<uintptr_t>(it.dst), it.rows * up16(it.len));
        g_operands[reinterpret_cast<uintptr_t>(it.dst)] = {reinterpret_cast<uintptr_t>(it.dst), it.rows, it.len,
                                                           up16(it.len)};
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
}  // namespace ns

int main()
{
    std::mt19937_64 rng(1);
    auto pick = [&](std::initializer_list<int64_t> v) { return v.begin()[rng() % v.size()]; };
    for (int round = 0; round < 3000; ++round) {
        const int op = (int)(rng() % 3);
        const int32_t dtype = op == NS_Q8_GRAD_INPUT ? NS_BF16 : (int32_t)(rng() % 2);
        const int n = (int)pick({1, 1, 2, 5, 41, 90});
        std::vector<ns_q8_layer> layers(n);
        g_operands.clear();
        g_taken.clear();
        g_written.clear();
        g_split.clear();
        uintptr_t at = 0x100000000;   // addresses are never followed
        auto place = [&](int64_t rows, int64_t cols, int64_t elt, int64_t* ld) -> uintptr_t {
            *ld = rows == 0 || rng() % 3 == 0 ? std::max<int64_t>(1, cols) : cols + (int64_t)(rng() % 40);
            if (rng() % 3)
                *ld = (*ld * elt + 15) / 16 * 16 / elt;
            uintptr_t p = at + (rng() % 4 ? 0 : elt * (rng() % 16));
            at += (uintptr_t)(rows * *ld * elt + 4096) / 4096 * 4096 + 4096;
            if (rows * cols == 0)
                return 0;
            g_operands[p] = {p, rows, cols * elt, *ld * elt};
            return p;
        };
        int64_t outputs = 0;
        for (ns_q8_layer& l : layers) {
            const int64_t most = n > 2 ? 700 : 5000;
            auto dim = [&] {
                return std::min<int64_t>(most, pick({0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200,
                                                     255, 256, 257, 500, 513, 1000, 2048, 2304, 4096, 5000}));
            };
            l = {};
            l.tokens = dim();
            l.out_features = dim();
            l.in_features = dim();
            const int64_t t = l.tokens, o = l.out_features, k = l.in_features;
            l.xq = reinterpret_cast<const int8_t*>(place(t, k, 1, &l.ld_xq));
            l.wq = reinterpret_cast<const int8_t*>(place(o, k, 1, &l.ld_wq));
            l.dy = reinterpret_cast<const void*>(place(t, o, 2, &l.ld_dy));
            l.x_scale = reinterpret_cast<const float*>(0x1000);
            l.w_scale = reinterpret_cast<const float*>(0x1000);
            const int64_t m = op == NS_Q8_GRAD_WEIGHT ? o : t, c = op == NS_Q8_MATMUL ? o : k;
            l.out = reinterpret_cast<void*>(place(m, c, dtype == NS_BF16 ? 2 : 4, &l.ld_out));
            outputs += m > 0 && c > 0;
        }
        size_t need = 0;
        EXPECT(ns_q8_workspace_bytes(op, layers.data(), n, dtype, &need) == NS_OK, "%s", ns::g_msg.c_str());
        g_ws = 0x7000000000;
        g_ws_end = g_ws + need;
        void* ws = reinterpret_cast<void*>(g_ws);
        const ns_status st = op == NS_Q8_MATMUL       ? ns_q8_matmul(layers.data(), n, dtype, ws, need, nullptr)
                             : op == NS_Q8_GRAD_INPUT ? ns_q8_grad_input(layers.data(), n, ws, need, nullptr)
                                                      : ns_q8_grad_weight(layers.data(), n, 0.5f, dtype, ws, need, nullptr);
        EXPECT(st == NS_OK, "%s", ns::g_msg.c_str());
        EXPECT((int64_t)g_written.size() == outputs, "every output written: %zu of %lld", g_written.size(),
               (long long)outputs);
        EXPECT(g_split.empty(), "a split product not joined");

        std::vector<ns_q8_rows> mats((size_t)pick({1, 3, 64, 65, 200}));
        for (ns_q8_rows& m : mats) {
            m.rows = pick({0, 1, 3, 4, 5, 300});
            m.cols = pick({0, 1, 7, 2048, 2049, 10240});
            m.values = reinterpret_cast<void*>(at);
            m.ld_values = std::max<int64_t>(1, m.cols);
            m.q = reinterpret_cast<int8_t*>(at + (64 << 20));
            m.ld_q = m.ld_values;
            m.scale = reinterpret_cast<float*>(at + (100 << 20));
            at += 256 << 20;
        }
        EXPECT(ns_q8_quantize(mats.data(), (int32_t)mats.size(), (int)(rng() % 2), dtype, nullptr) == NS_OK, "%s",
               ns::g_msg.c_str());
        EXPECT(ns_q8_dequantize(mats.data(), (int32_t)mats.size(), dtype, nullptr) == NS_OK, "%s", ns::g_msg.c_str());
    }
    if (g_fail)
        return 1;
    std::printf("q8_check ok\n");
    return 0;
}
