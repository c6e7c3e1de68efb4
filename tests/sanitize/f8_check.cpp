// The host code of the 8-bit floating-point layers and of the experts' router under
// AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_f8_sanitizers.py builds
// this with g++, ns_f8_api.cpp and ns_route_api.cpp). The kernel launchers below only
// look at what they are given: random lists, and for every launch
//   - each item's workgroups follow the previous item's, and cover its output;
//   - the blocks of k of a split product are covered once by its pieces;
//   - pieces lie inside the workspace, apart from one another, and are joined;
//   - the buffer resources that the product kernels build end with the operands
//     (rounded up to 16 bytes), and their offsets fit 31 bits;
//   - ranges of a matrix's rows are whole blocks, and cover it once.
// Prints "f8_check ok" and returns 0 when everything holds.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_enqueue.h"
#include "ns_f8.h"
#include "ns_route.h"

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

struct Operand { int64_t rows, cols, ld; };
std::map<uintptr_t, Operand> g_operands;
std::vector<std::pair<uintptr_t, uintptr_t>> g_taken;   // of the workspace
uintptr_t g_ws, g_ws_end;
std::map<uintptr_t, int> g_written;                     // outputs, by address
std::map<uintptr_t, int> g_split;                       // of them, still to be joined
std::map<uintptr_t, int64_t> g_rows;                    // rows of a matrix done so far, by address
int g_dtype;

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

void take(uintptr_t at, int64_t n)
{
    EXPECT(at % 16 == 0 && at >= g_ws && at + n <= g_ws_end, "outside the workspace");
    for (auto& p : g_taken)
        EXPECT(at >= p.second || at + n <= p.first, "workspace used twice");
    g_taken.push_back({at, at + n});
}

void check_product(const ns::F8Item& it, int bm, int bn)
{
    for (int side = 0; side < 2; ++side) {
        const char* p = side ? it.b : it.a;
        auto o = g_operands.find(reinterpret_cast<uintptr_t>(p));
        EXPECT(o != g_operands.end(), "an operand that is none");
        if (o == g_operands.end())
            return;
        const int64_t rows = side ? it.n : it.m, ld = side ? it.ldb : it.lda, tile = std::min<int64_t>(rows, side ? bn : bm);
        EXPECT(o->second.rows == rows && o->second.cols == it.k && o->second.ld == ld, "an operand's sizes");
        EXPECT(ld % 16 == 0 && ld >= up16(it.k), "a pitch that the loads pass");
        // the furthest row that a tile addresses, past the end of the operand or not
        EXPECT((side ? bn : bm) * ld < (int64_t(1) << 31) && (tile - 1) * ld + up16(it.k) < (int64_t(1) << 31), "offsets");
    }
    const int64_t elt = g_dtype == NS_BF16 ? 2 : 4;
    EXPECT((bm * (int64_t)it.ldo + bn) * elt < (int64_t(1) << 31) + bm * elt, "an output's offsets");
    EXPECT((bm * (int64_t)it.n + bn) * 4 <= (int64_t(1) << 31) || it.nsplit == 1, "a piece's offsets");
    EXPECT(g_written[reinterpret_cast<uintptr_t>(it.out)]++ == 0, "an output written twice");
}

hipError_t tiles(const ns::F8Batch& b, int nwg, int bm, int bn, bool may_split)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= ns::kF8Items, "items");
    for (int i = 0; i < b.count; ++i) {
        const ns::F8Item& it = b.it[i];
        const int blocks = (it.k + ns::kF8Block - 1) / ns::kF8Block;
        EXPECT(it.begin == at && it.m > ns::kF8Few && it.k > 0, "an item");
        EXPECT(it.ntn == (it.n + bn - 1) / bn, "ntn");
        EXPECT(it.nsplit >= 1 && (may_split || it.nsplit == 1), "nsplit");
        EXPECT((int64_t)it.nsplit * it.per >= blocks && (int64_t)(it.nsplit - 1) * it.per < blocks,
               "pieces cover the blocks, none empty");
        at += (int64_t)((it.m + bm - 1) / bm) * it.ntn * it.nsplit;
        check_product(it, bm, bn);
        if (it.nsplit > 1) {
            take(reinterpret_cast<uintptr_t>(it.part), (int64_t)it.nsplit * it.m * it.n * 4);
            g_split[reinterpret_cast<uintptr_t>(it.out)] = it.nsplit;
        }
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}

// A range of a matrix's rows: it begins where the last one of that matrix ended.
void range(uintptr_t values, int64_t ld_bytes, int64_t rows)
{
    auto m = std::prev(g_rows.upper_bound(values));
    EXPECT(values == m->first + (uintptr_t)(m->second * ld_bytes), "a range that does not follow the last");
    EXPECT(m->second % ns::kF8Block == 0, "a range that cuts a block");
    m->second += rows;
}

}  // namespace

namespace ns {
hipError_t launch_f8_quantize(const F8RowsBatch& b, int nwg, int, int, int dtype, hipStream_t)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= kF8RowsItems && nwg < 1 << 24, "items");
    for (int i = 0; i < b.count; ++i) {
        const F8RowsItem& it = b.it[i];
        EXPECT(it.begin == at && it.ntn == (it.cols + 127) / 128, "an item");
        at += (int64_t)((it.rows + 127) / 128) * it.ntn;
        range(reinterpret_cast<uintptr_t>(it.values), it.ldv * (dtype == NS_BF16 ? 2 : 4), it.rows);
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_f8_dequantize(const F8ValuesBatch& b, int nwg, int dtype, hipStream_t)
{
    int64_t at = 0;
    const int64_t elt = dtype == NS_BF16 ? 2 : 4;
    EXPECT(b.count > 0 && b.count <= kF8ValuesItems && nwg < 1 << 24, "items");
    for (int i = 0; i < b.count; ++i) {
        const F8ValuesItem& it = b.it[i];
        EXPECT(it.begin == at, "begin");
        // what the kernel takes from it: g pieces a row, rows together or one in parts
        const int64_t g = (it.cols * elt + 15) / 16, n = kF8ValuesPieces;
        const int64_t wgs = f8_values_wgs(it.rows, it.cols, elt);
        EXPECT(g <= n ? wgs * (n / g) >= it.rows && (wgs - 1) * (n / g) < it.rows : wgs % it.rows == 0 && wgs / it.rows * n >= g,
               "pieces");
        at += wgs;
        range(reinterpret_cast<uintptr_t>(it.values), it.ldv * elt, it.rows);
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_f8_small(const F8Batch& b, int nwg, int, int, int, hipStream_t) { return tiles(b, nwg, kF8SmallM, kF8SmallN, true); }
hipError_t launch_f8_mid(const F8Batch& b, int nwg, int, int, int, hipStream_t) { return tiles(b, nwg, kF8MidM, kF8MidN, false); }
hipError_t launch_f8_big(const F8Batch& b, int nwg, int, int dtype, hipStream_t)
{
    for (int i = 0; i < b.count; ++i) {
        const F8Item& it = b.it[i];
        EXPECT((it.flags & 3) == 3 && it.n % 4 == 0 && it.ldo % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(it.out) % (dtype == NS_BF16 ? 8 : 16) == 0, "not for large tiles");
    }
    return tiles(b, nwg, kF8Big, kF8Big, false);
}
hipError_t launch_f8_few(const F8Batch& b, int nwg, int rows, int, int, int, hipStream_t)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= kF8Items && (rows == 16 || rows == 32), "items");
    for (int i = 0; i < b.count; ++i) {
        const F8Item& it = b.it[i];
        EXPECT(it.begin == at && it.m <= kF8Few && it.nsplit == 1 && it.k > 0, "few rows");
        at += (it.n + rows - 1) / rows;
        check_product(it, kF8Few, rows);
    }
    EXPECT(at == nwg, "workgroups");
    return hipSuccess;
}
hipError_t launch_f8_join(const F8Batch& b, int nwg, int, hipStream_t)
{
    int64_t at = 0;
    for (int i = 0; i < b.count; ++i) {
        const F8Item& it = b.it[i];
        EXPECT(it.begin == at, "begin");
        at += ((int64_t)it.m * it.n + kF8JoinElems - 1) / kF8JoinElems;
        if (it.nsplit == 0) {
            EXPECT(it.k == 0 && g_written[reinterpret_cast<uintptr_t>(it.out)]++ == 0, "an output written twice");
            continue;
        }
        auto s = g_split.find(reinterpret_cast<uintptr_t>(it.out));
        EXPECT(s != g_split.end() && s->second == it.nsplit, "joins what was split");
        if (s != g_split.end())
            g_split.erase(s);
    }
    EXPECT(at == nwg && nwg < 1 << 24, "workgroups");
    return hipSuccess;
}

static int64_t g_routed, g_groups;
hipError_t launch_route(const RouteArgs& a, int nwg, int, hipStream_t)
{
    g_groups = nwg;
    ++g_routed;
    EXPECT(nwg >= 1 && nwg <= kRouteGroups, "workgroups");
    if (nwg == 1)
        return hipSuccess;
    const int64_t n = (int64_t)nwg * ((a.experts + kRouteJoin - 1) / kRouteJoin * kRouteJoin) * 4;
    g_taken.clear();
    take(reinterpret_cast<uintptr_t>(a.part_probs), n);
    take(reinterpret_cast<uintptr_t>(a.part_counts), n);
    EXPECT(reinterpret_cast<uintptr_t>(a.part_routed) >= g_taken[1].second &&
               reinterpret_cast<uintptr_t>(a.arrived) >= reinterpret_cast<uintptr_t>(a.part_routed) + nwg * 4 &&
               reinterpret_cast<uintptr_t>(a.arrived) + 4 <= g_ws_end, "the small parts");
    return hipSuccess;
}
hipError_t launch_route_join(const RouteArgs&, int nwg, hipStream_t)
{
    EXPECT(nwg == g_groups && nwg > 1, "joins what was routed");
    return hipSuccess;
}
hipError_t launch_route_grad(const RouteGradArgs& a, int nwg, int, hipStream_t)
{
    EXPECT(nwg >= 1 && nwg <= 2048 && a.tokens > 0 && (int64_t)(nwg - 1) * route_tokens(a.experts) < a.tokens, "workgroups");
    return hipSuccess;
}
}  // namespace ns

int main()
{
    std::mt19937_64 rng(1);
    auto pick = [&](std::initializer_list<int64_t> v) { return v.begin()[rng() % v.size()]; };
    uintptr_t at = 0;
    // (addresses are never followed)
    auto place = [&](int64_t bytes) {
        const uintptr_t p = at;
        at += (uintptr_t)(bytes + 4096) / 4096 * 4096 + 4096;
        return p;
    };
    for (int round = 0; round < 3000; ++round) {
        const int32_t dtype = g_dtype = (int32_t)(rng() % 2);
        const int64_t elt = dtype == NS_BF16 ? 2 : 4;
        at = 0x100000000;
        g_operands.clear();
        g_taken.clear();
        g_written.clear();
        g_split.clear();
        std::vector<ns_f8_product> products((size_t)pick({1, 1, 2, 5, 37, 90}));
        const int64_t most = products.size() > 2 ? 700 : 9000;
        auto dim = [&] {
            return std::min(most, pick({0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 500,
                                        513, 1000, 2048, 2304, 4096, 5000, 8192, 9000}));
        };
        auto matrix = [&](int64_t rows, int64_t cols) {
            ns_f8_matrix m{};
            m.rows = rows;
            m.cols = cols;
            m.format = 0;
            m.scale_type = rng() % 3 ? NS_F8_SCALE_POW2 : NS_F8_SCALE_FP32;
            m.square = (int32_t)(rng() % 2);
            m.ld_q = up16(std::max<int64_t>(1, cols)) + 16 * (int64_t)(rng() % 3);
            if (rng() % 200 == 0)
                m.ld_q = int64_t(1) << 21;
            m.ld_scale = up16(std::max<int64_t>(1, m.square ? (rows + 127) / 128 : rows));
            const uintptr_t q = place(rows * m.ld_q);
            m.q = reinterpret_cast<void*>(rows && cols ? q : 0);
            m.scale = reinterpret_cast<void*>(rows && cols ? place((cols + 127) / 128 * m.ld_scale * 4) : 0);
            g_operands[q] = {rows, cols, m.ld_q};
            return m;
        };
        int64_t outputs = 0;
        for (ns_f8_product& p : products) {
            const int64_t m = dim(), n = dim(), k = dim();
            p.a = matrix(m, k);
            p.a.format = (int32_t)(rng() % 2);
            p.b = matrix(n, k);
            p.ld_out = std::max<int64_t>(1, n) + (rng() % 2 ? 0 : (int64_t)(rng() % 9));
            if (rng() % 100 == 0)
                p.ld_out = int64_t(1) << 21;
            p.out = reinterpret_cast<void*>(place(m * p.ld_out * elt) + (rng() % 3 ? 0 : elt * (rng() % 5)));
            outputs += m > 0 && n > 0;
        }
        const int32_t count = (int32_t)products.size();
        size_t need = 0;
        EXPECT(ns_f8_workspace_bytes(products.data(), count, dtype, &need) == NS_OK, "%s", ns::g_msg.c_str());
        g_ws = 0x700000000000;
        g_ws_end = g_ws + need;
        if (need) {
            EXPECT(ns_f8_matmul(products.data(), count, 0.5f, dtype, reinterpret_cast<void*>(g_ws), need - 1, nullptr) ==
                       NS_EINVAL && g_written.empty(), "a workspace too small");
        }
        EXPECT(ns_f8_matmul(products.data(), count, 0.5f, dtype, reinterpret_cast<void*>(g_ws), need, nullptr) == NS_OK,
               "%s", ns::g_msg.c_str());
        EXPECT((int64_t)g_written.size() == outputs, "every output written: %zu of %lld", g_written.size(),
               (long long)outputs);
        EXPECT(g_split.empty(), "a split product not joined");

        for (int back = 0; back < 2; ++back) {
            std::vector<ns_f8_rows> rows((size_t)pick({1, 3, 40, 41, 100}));
            std::vector<ns_f8_values> vals(rows.size());
            const int32_t square = (int32_t)(rng() % 2), type = (int32_t)(rng() % 2);
            g_rows.clear();
            std::map<uintptr_t, int64_t> want;
            for (size_t i = 0; i < rows.size(); ++i) {
                ns_f8_rows& m = rows[i];
                const bool huge = rng() % 300 == 0;
                m.rows = huge ? pick({1 << 24, (1 << 24) - 1}) : pick({0, 1, 3, 127, 128, 129, 300, 5000});
                m.cols = huge ? pick({1, 130, 70000, 1 << 24}) : pick({0, 1, 7, 128, 129, 2049, 10240, 1 << 20});
                m.ld_values = std::max<int64_t>(1, m.cols) + (int64_t)(rng() % 5);
                m.values = reinterpret_cast<void*>(place(m.rows * m.ld_values * elt));
                m.ld_q = up16(std::max<int64_t>(1, m.cols));
                m.q = reinterpret_cast<void*>(place(m.rows * m.ld_q));
                m.ld_scale = up16(std::max<int64_t>(1, square ? (m.rows + 127) / 128 : m.rows));
                m.scale = reinterpret_cast<void*>(place((m.cols + 127) / 128 * m.ld_scale * 4));
                m.ld_qt = up16(std::max<int64_t>(1, m.rows));
                m.qt = rng() % 2 ? nullptr : reinterpret_cast<void*>(place(m.cols * m.ld_qt));
                m.ld_scale_t = up16(std::max<int64_t>(1, square ? (m.cols + 127) / 128 : m.cols));
                m.scale_t = m.qt ? reinterpret_cast<void*>(place((m.rows + 127) / 128 * m.ld_scale_t * 4)) : nullptr;
                ns_f8_values& v = vals[i];
                v = ns_f8_values{};
                v.matrix.rows = m.rows;
                v.matrix.cols = m.cols;
                v.matrix.q = m.q;
                v.matrix.ld_q = m.ld_q;
                v.matrix.scale = m.scale;
                v.matrix.ld_scale = m.ld_scale;
                v.matrix.scale_type = type;
                v.matrix.square = square;
                v.values = const_cast<void*>(m.values);
                v.ld_values = m.ld_values;
                if (m.rows && m.cols) {
                    g_rows[reinterpret_cast<uintptr_t>(m.values)] = 0;
                    want[reinterpret_cast<uintptr_t>(m.values)] = m.rows;
                }
            }
            const ns_status st = back ? ns_f8_dequantize(vals.data(), (int32_t)vals.size(), dtype, nullptr)
                                      : ns_f8_quantize(rows.data(), (int32_t)rows.size(), 0, type, square, dtype, nullptr);
            EXPECT(st == NS_OK, "%s", ns::g_msg.c_str());
            EXPECT(g_rows == want, "rows of a matrix left out");
        }

        ns_route r{};
        r.tokens = pick({0, 1, 31, 32, 33, 128, 129, 1000, 16384, 16385, 1 << 24});
        r.experts = pick({1, 16, 17, 255, 256, 257, 512, 1000, 1024});
        r.ld = r.experts + (int64_t)(rng() % 3);
        r.top_k = (int32_t)std::min<int64_t>(r.experts, pick({1, 2, 16}));
        void* const some = reinterpret_cast<void*>(0x1000);
        r.logits = some;
        r.chosen = r.counts = r.routed = static_cast<int32_t*>(some);
        r.weights = r.probs = r.loss = static_cast<float*>(some);
        EXPECT(ns_route_workspace_bytes(r.tokens, r.experts, &need) == NS_OK, "%s", ns::g_msg.c_str());
        EXPECT(r.tokens > 32 || need == 0, "a workspace for few tokens");
        g_ws_end = g_ws + need;
        EXPECT(ns_route_experts(&r, dtype, reinterpret_cast<void*>(g_ws), need, nullptr) == NS_OK, "%s", ns::g_msg.c_str());
        ns_route_grad g{};
        g.tokens = r.tokens;
        g.experts = r.experts;
        g.logits = g.out = some;
        g.ld = g.ld_out = r.ld;
        g.top_k = r.top_k;
        g.chosen = g.counts = g.routed = static_cast<const int32_t*>(some);
        g.dweights = g.dloss = static_cast<const float*>(some);
        EXPECT(ns_route_experts_grad(&g, dtype, nullptr) == NS_OK, "%s", ns::g_msg.c_str());
    }
    EXPECT(ns::g_routed == 3000, "routed");
    if (g_fail)
        return 1;
    std::printf("f8_check ok\n");
    return 0;
}
