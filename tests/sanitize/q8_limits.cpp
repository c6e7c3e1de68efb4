// The host code of the 8-bit linear layers at the largest sizes it takes
// (tests/test_q8_limits.py builds this with g++, the sanitizers and
// ns_q8_api.cpp; no address is followed). HIP launches fewer than 2^32 threads
// at once. The launchers below check that, and that the parts a matrix comes in
// follow one another and cover it. Prints "q8_limits ok" when everything holds.
#include <cstdio>
#include <cstdlib>
#include <map>
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

int g_launches = 0;
void launch(int64_t nwg, int threads)
{
    ++g_launches;
    EXPECT(nwg > 0 && nwg * threads < (int64_t(1) << 32), "%lld workgroups of %d threads", (long long)nwg, threads);
}

// A matrix that arrives in ranges of rows: by the address after the last one.
struct Whole { uintptr_t base; int64_t rows, pitch, done; };   // pitch: bytes
std::vector<Whole> g_whole;
Whole* next_rows(const void* p, int64_t rows)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    for (Whole& w : g_whole)
        if (w.done < w.rows && w.base + (uintptr_t)(w.done * w.pitch) == at) {
            EXPECT(rows > 0 && w.done + rows <= w.rows, "more rows than there are");
            w.done += rows;
            return &w;
        }
    EXPECT(false, "rows that do not follow");
    return nullptr;
}
void all_covered()
{
    for (const Whole& w : g_whole)
        EXPECT(w.done == w.rows, "%lld of %lld rows", (long long)w.done, (long long)w.rows);
}

template <typename B, typename F>
void items(const B& b, int most, int64_t nwg, F&& groups)
{
    int64_t at = 0;
    EXPECT(b.count > 0 && b.count <= most, "items");
    for (int i = 0; i < b.count; ++i) {
        EXPECT(b.it[i].begin == at, "begin");
        at += groups(b.it[i]);
    }
    EXPECT(at == nwg, "workgroups");
}

constexpr uintptr_t kQ = 0x100000000000, kScale = 0x200000000000;   // beside values
hipError_t rows_launch(const ns::Q8RowsBatch& b, int nwg, int elt)
{
    launch(nwg, 256);
    items(b, ns::kQ8RowsItems, nwg, [&](const ns::Q8RowsItem& it) {
        Whole* w = next_rows(it.values, it.rows);
        if (w) {
            const int64_t row = w->done - it.rows;
            EXPECT(it.ldv * elt == w->pitch, "pitch");
            EXPECT(reinterpret_cast<uintptr_t>(it.q) == w->base + kQ + (uintptr_t)(row * it.ldq), "q's rows");
            EXPECT(reinterpret_cast<uintptr_t>(it.scale) == w->base + kScale + 4 * (uintptr_t)row, "scales");
        }
        const int per = ns::q8_rows_per_wg(it.cols);
        return ((int64_t)it.rows + per - 1) / per;
    });
    return hipSuccess;
}
int g_elt;
std::vector<int> g_big;   // layers, workgroups and whole tiles of the last launch of large tiles

}  // namespace

namespace ns {
hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int, hipStream_t) { return rows_launch(b, nwg, g_elt); }
hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int, hipStream_t) { return rows_launch(b, nwg, g_elt); }
static hipError_t tiles(const Q8Batch& b, int64_t nwg, int edge)
{
    items(b, kQ8Items, nwg, [&](const Q8Item& it) {
        return (int64_t)((it.m + edge - 1) / edge) * ((it.n + edge - 1) / edge) * it.nsplit;
    });
    return hipSuccess;
}
hipError_t launch_q8_big(int, const Q8Batch& b, int nwg, int nwhole, int, hipStream_t)
{
    launch(nwg, 256);
    g_big = {b.count, nwg, nwhole};
    return tiles(b, nwhole + (nwg - nwhole) / 2, kQ8Big);
}
hipError_t launch_q8_mid(int, const Q8Batch& b, int nwg, int, hipStream_t)
{
    launch(nwg, 256);
    return tiles(b, nwg, kQ8Mid);
}
hipError_t launch_q8_thin(const Q8Batch& b, int nwg, int, hipStream_t)
{
    launch(nwg, 256);
    items(b, kQ8Items, nwg, [&](const Q8Item& it) { return (int64_t)it.ntn * it.nsplit; });
    return hipSuccess;
}
hipError_t launch_q8_few(const Q8Batch& b, int nwg, int, hipStream_t)
{
    launch(nwg, 512);
    items(b, kQ8Items, nwg, [&](const Q8Item& it) {
        return (int64_t)(it.n + q8_few_channels(it.m) - 1) / q8_few_channels(it.m);
    });
    return hipSuccess;
}
hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int, hipStream_t)
{
    launch(nwg, 256);
    items(b, kQ8Items, nwg, [&](const Q8Item& it) {
        if (it.nsplit == 0) {
            Whole* w = next_rows(it.out, it.m);
            if (w && op == kQ8Matmul)
                EXPECT(reinterpret_cast<uintptr_t>(it.sa) == w->base + kScale + 4 * (uintptr_t)(w->done - it.m),
                       "scales");
        }
        return ((int64_t)it.m * it.n + kQ8JoinElems - 1) / kQ8JoinElems;
    });
    return hipSuccess;
}
hipError_t launch_q8_align(const Q8AlignBatch& b, int nwg, hipStream_t)
{
    launch(nwg, 256);
    items(b, kQ8AlignItems, nwg, [&](const Q8AlignItem& it) {
        Whole* w = next_rows(it.src, it.rows);
        const int64_t len = (it.len + 15) / 16 * 16;
        if (w) {
            static std::map<uintptr_t, uintptr_t> copy;   // a copy's first row
            const int64_t row = w->done - it.rows;
            if (row == 0)
                copy[w->base] = reinterpret_cast<uintptr_t>(it.dst);
            EXPECT(it.pitch == w->pitch && reinterpret_cast<uintptr_t>(it.dst) == copy[w->base] + (uintptr_t)(row * len),
                   "the copy's rows");
        }
        return (it.rows * (len / 16) + kQ8AlignChunks - 1) / kQ8AlignChunks;
    });
    return hipSuccess;
}
}  // namespace ns

int main()
{
    const int64_t most = int64_t(1) << 24;
    // rows to 8 bits and back: tall matrices of short and of long rows, many of
    // them, sums that end at the limit and just beside it
    struct { int64_t count, rows, cols; } rows[] = {{4, most, 8}, {3, most, 8}, {1, most, 2049}, {2, most - 1, 4096},
                                                    {64, most, 1}, {70, (1 << 18) + 3, 3000}, {17, 1 << 20, 2049},
                                                    {16, 1 << 20, 2049}, {100, 5, 7}};
    for (auto& r : rows)
        for (int dtype : {NS_BF16, NS_FP32}) {
            g_elt = dtype == NS_BF16 ? 2 : 4;
            std::vector<ns_q8_rows> mats;
            for (int back : {0, 1}) {
                g_whole.clear();
                mats.clear();
                uintptr_t at = 0x10000000;
                for (int64_t i = 0; i < r.count; ++i) {
                    const int64_t ld = r.cols + i % 3;
                    mats.push_back({r.rows, r.cols, reinterpret_cast<void*>(at), ld,
                                    reinterpret_cast<int8_t*>(at + kQ), ld, reinterpret_cast<float*>(at + kScale)});
                    g_whole.push_back({at, r.rows, ld * g_elt, 0});
                    at += (uintptr_t)(r.rows * ld * 8 + 4096);
                }
                const ns_status st = back ? ns_q8_dequantize(mats.data(), (int32_t)r.count, dtype, nullptr)
                                          : ns_q8_quantize(mats.data(), (int32_t)r.count, 0, dtype, nullptr);
                EXPECT(st == NS_OK, "%s", ns::g_msg.c_str());
                all_covered();
            }
        }
    // products: sums over nothing in large outputs, operands copied to aligned
    // rows, outputs of many tiles, few rows, few tokens
    struct { int op; int64_t count, tokens, out, in, extra; bool whole_out; } products[] = {
        {NS_Q8_GRAD_WEIGHT, 1, 0, most, 1024, 0, true}, {NS_Q8_GRAD_WEIGHT, 3, 0, most, 2048, 0, true},
        {NS_Q8_MATMUL, 1, most, 2048, 0, 0, true},      {NS_Q8_GRAD_INPUT, 1, most, 0, 1500, 0, true},
        {NS_Q8_GRAD_INPUT, 1, most, 2047, 40, 1, false}, {NS_Q8_GRAD_WEIGHT, 1, most, 2047, 100, 1, false},
        {NS_Q8_MATMUL, 1, most, 100, 4001, 1, false},    {NS_Q8_MATMUL, 41, most, 400, 64, 0, false},
        {NS_Q8_GRAD_INPUT, 40, most, 64, 512, 0, false}, {NS_Q8_GRAD_WEIGHT, 40, most, 64, 2048, 0, false},
        {NS_Q8_MATMUL, 90, 32, 1 << 21, 16, 0, false},   {NS_Q8_MATMUL, 90, 1, 1 << 21, 16, 0, false}};
    for (auto& c : products) {
        g_whole.clear();
        std::vector<ns_q8_layer> layers;
        uintptr_t at = 0x10000000;
        for (int64_t i = 0; i < c.count; ++i) {
            // `extra`: rows at pitches that are no multiple of 16 bytes
            auto ld = [&](int64_t cols, int64_t unit) { return (cols + unit - 1) / unit * unit + c.extra; };
            ns_q8_layer l{};
            l.tokens = c.tokens, l.out_features = c.out, l.in_features = c.in;
            l.ld_xq = l.ld_wq = ld(c.in, 16), l.ld_dy = ld(c.out, 8);
            const int64_t m = c.op == NS_Q8_GRAD_WEIGHT ? c.out : c.tokens, n = c.op == NS_Q8_MATMUL ? c.out : c.in;
            auto place = [&](int64_t rows, int64_t pitch, bool checked) {
                const uintptr_t p = at;
                at += (uintptr_t)(rows * pitch + 4096) / 4096 * 4096;
                if (checked)
                    g_whole.push_back({p, rows, pitch, 0});
                return p;
            };
            const bool copy = c.extra > 0;
            l.xq = reinterpret_cast<int8_t*>(place(c.tokens, l.ld_xq, copy && c.op != NS_Q8_GRAD_INPUT));
            l.wq = reinterpret_cast<int8_t*>(place(c.out, l.ld_wq, copy && c.op != NS_Q8_GRAD_WEIGHT));
            l.dy = reinterpret_cast<void*>(place(c.tokens, 2 * l.ld_dy, copy && c.op != NS_Q8_MATMUL));
            l.ld_out = (n + 7) / 8 * 8;
            l.out = reinterpret_cast<void*>(place(m, 2 * l.ld_out, c.whole_out));
            l.x_scale = l.w_scale = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(l.out) + kScale);
            layers.push_back(l);
        }
        size_t need = 0;
        const int32_t n = (int32_t)c.count;
        EXPECT(ns_q8_workspace_bytes(c.op, layers.data(), n, NS_BF16, &need) == NS_OK, "%s", ns::g_msg.c_str());
        void* ws = reinterpret_cast<void*>(0x400000000000);
        const ns_status st = c.op == NS_Q8_MATMUL       ? ns_q8_matmul(layers.data(), n, NS_BF16, ws, need, nullptr)
                             : c.op == NS_Q8_GRAD_INPUT ? ns_q8_grad_input(layers.data(), n, ws, need, nullptr)
                                                        : ns_q8_grad_weight(layers.data(), n, 0.5f, NS_BF16, ws, need,
                                                                            nullptr);
        EXPECT(st == NS_OK, "%s", ns::g_msg.c_str());
        all_covered();
    }
    // a list of layers that share large tiles, each too small to have them alone:
    // 334 tiles, the 78 behind the first 256 as halves
    const int64_t shapes[][3] = {{2560, 2560, 1600}, {2040, 2550, 2101}, {2048, 2048, 1537}, {1270, 2555, 3000},
                                 {2048, 1280, 1555}};
    for (int op : {NS_Q8_MATMUL, NS_Q8_GRAD_INPUT, NS_Q8_GRAD_WEIGHT})
        for (int alone : {0, 1}) {
            std::vector<ns_q8_layer> layers;
            uintptr_t at = 0x10000000;
            for (auto& s : shapes) {
                ns_q8_layer l{};
                l.tokens = op == NS_Q8_GRAD_WEIGHT ? s[2] : s[0];
                l.out_features = op == NS_Q8_MATMUL ? s[1] : op == NS_Q8_GRAD_INPUT ? s[2] : s[0];
                l.in_features = op == NS_Q8_MATMUL ? s[2] : s[1];
                l.ld_xq = l.ld_wq = l.ld_dy = l.ld_out = 4096;
                l.xq = l.wq = reinterpret_cast<int8_t*>(0x1000);
                l.dy = reinterpret_cast<void*>(0x1000);
                l.x_scale = l.w_scale = reinterpret_cast<float*>(0x1000);
                l.out = reinterpret_cast<void*>(at);
                at += 1 << 26;
                layers.push_back(l);
            }
            g_big.clear();
            for (int32_t i = 0; i < (alone ? 5 : 1); ++i) {
                const int32_t n = alone ? 1 : 5;
                const ns_status st =
                    op == NS_Q8_MATMUL       ? ns_q8_matmul(&layers[i], n, NS_FP32, nullptr, 0, nullptr)
                    : op == NS_Q8_GRAD_INPUT ? ns_q8_grad_input(&layers[i], n, nullptr, 0, nullptr)
                                             : ns_q8_grad_weight(&layers[i], n, 0.5f, NS_FP32, nullptr, 0, nullptr);
                EXPECT(st == NS_OK, "%s", ns::g_msg.c_str());
            }
            EXPECT(g_big == (alone ? std::vector<int>{} : std::vector<int>{5, 412, 256}), "large tiles, op %d", op);
        }
    EXPECT(g_launches > 0, "no launch");
    if (g_fail)
        return 1;
    std::printf("q8_limits ok\n");
    return 0;
}
