// Which kernel each product of a list goes to (tests/test_f8_kinds.py builds this with
// g++ and ns_f8_api.cpp, no device code). Reads lists from stdin:
//   dtype count, then `count` times: m n k fp32_scales square offset ld_out
// (offset: bytes by which the output is off an aligned address) and prints for each one
//   the workspace, then `kind pieces` of every product in turn.
#include <cstdint>
#include <cstdio>
#include <map>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_enqueue.h"
#include "ns_f8.h"

namespace ns {
ns_status fail(ns_status s, const std::string& msg)
{
    std::fprintf(stderr, "%s\n", msg.c_str());
    return s;
}
ns_status hip_fail(hipError_t, const char* what) { return fail(NS_EHIP, what); }
void clear_error() {}

static std::map<const void*, std::string> g_kind;
static hipError_t note(const char* kind, const F8Batch& b)
{
    for (int i = 0; i < b.count; ++i)
        g_kind[b.it[i].out] += (g_kind[b.it[i].out].empty() ? "" : "+") + (kind + (" " + std::to_string(b.it[i].nsplit)));
    return hipSuccess;
}
hipError_t launch_f8_quantize(const F8RowsBatch&, int, int, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_dequantize(const F8ValuesBatch&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_small(const F8Batch& b, int, int, int, int, hipStream_t) { return note("small", b); }
// (the combinations that the library has mid tiles of)
hipError_t launch_f8_mid(const F8Batch& b, int, int, int any, int dtype, hipStream_t)
{
    return note((dtype == NS_FP32) == (any != 0) ? "mid" : "mid-that-there-is-not", b);
}
hipError_t launch_f8_big(const F8Batch& b, int, int, int dtype, hipStream_t)
{
    for (int i = 0; i < b.count; ++i)
        if (b.it[i].n % 4 || b.it[i].ldo % 4 || reinterpret_cast<uintptr_t>(b.it[i].out) % (dtype == NS_BF16 ? 8 : 16))
            return note("big-that-cannot-be", b);
    return note("big", b);
}
hipError_t launch_f8_few(const F8Batch& b, int, int, int, int, int, hipStream_t) { return note("few", b); }
hipError_t launch_f8_join(const F8Batch& b, int, int, hipStream_t)
{
    for (int i = 0; i < b.count; ++i)
        if (b.it[i].nsplit == 0)
            g_kind[b.it[i].out] = "none 0";
    return hipSuccess;
}
}  // namespace ns

int main()
{
    int dtype, count;
    while (std::scanf("%d %d", &dtype, &count) == 2) {
        std::vector<ns_f8_product> list((size_t)count);
        uintptr_t at = uintptr_t(1) << 40;   // (addresses are never followed)
        for (ns_f8_product& p : list) {
            long long m, n, k, any, square, offset, ld;
            if (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &m, &n, &k, &any, &square, &offset, &ld) != 7)
                return 1;
            auto matrix = [&](int64_t rows, bool sq) {
                ns_f8_matrix x{};
                x.rows = rows;
                x.cols = k;
                x.ld_q = (k + 15) / 16 * 16 + (k == 0) * 16;
                x.scale_type = any ? NS_F8_SCALE_FP32 : NS_F8_SCALE_POW2;
                x.square = sq;
                x.ld_scale = (rows + 15) / 16 * 16;
                x.q = reinterpret_cast<void*>(at += uintptr_t(1) << 36);
                x.scale = reinterpret_cast<void*>(at += uintptr_t(1) << 36);
                return x;
            };
            p = ns_f8_product{};
            p.a = matrix(m, false);
            p.b = matrix(n, square != 0);
            p.out = reinterpret_cast<void*>((at += uintptr_t(1) << 36) + (uintptr_t)offset);
            p.ld_out = ld;
        }
        size_t need = 0;
        if (ns_f8_workspace_bytes(list.data(), count, dtype, &need) != NS_OK)
            return 1;
        ns::g_kind.clear();
        if (ns_f8_matmul(list.data(), count, 0.f, dtype, reinterpret_cast<void*>(uintptr_t(1) << 36), need, nullptr) != NS_OK)
            return 1;
        std::printf("%zu", need);
        for (const ns_f8_product& p : list)
            std::printf(" %s", ns::g_kind[p.out].c_str());
        std::printf("\n");
    }
    return 0;
}
