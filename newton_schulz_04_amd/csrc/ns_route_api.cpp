// ns_route_api.cpp -- the C ABI of the experts' router (include/ns.h, ns_route_*):
// checks the arguments on the host and enqueues the kernels of ns_route.hip on the
// caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <limits>
#include <string>

#include "ns.h"
#include "ns_check.h"
#include "ns_enqueue.h"
#include "ns_route.h"

namespace {

using namespace ns;

ns_status check_sizes(int64_t tokens, int64_t experts)
{
    if (tokens < 0 || tokens > kMaxDim)
        return fail(NS_EINVAL, "tokens must be 0 .. 2^24");
    if (experts < 1 || experts > NS_ROUTE_MAX_EXPERTS)
        return fail(NS_EINVAL, "experts must be 1 .. " + std::to_string(NS_ROUTE_MAX_EXPERTS));
    return NS_OK;
}

ns_status check_pointer(const char* name, const void* p, size_t elt, bool needed)
{
    if (!p && needed)
        return fail(NS_EINVAL, std::string(name) + " must not be NULL");
    if (reinterpret_cast<uintptr_t>(p) % elt)
        return fail(NS_EINVAL, std::string(name) + " is not aligned to its element size");
    return NS_OK;
}

// What both calls share: sizes, the logits, the choice.
template <typename R>
ns_status check_common(const R* r, int32_t dtype)
{
    if (!r)
        return fail(NS_EINVAL, "the argument block must not be NULL");
    if (dtype != NS_BF16 && dtype != NS_FP32)
        return fail(NS_EDTYPE, "unknown dtype " + std::to_string(dtype));
    ns_status st;
    if ((st = check_sizes(r->tokens, r->experts)) != NS_OK)
        return st;
    if (r->top_k < 1 || r->top_k > NS_ROUTE_MAX_K || r->top_k > r->experts)
        return fail(NS_EINVAL, "top_k must be 1 .. " + std::to_string(NS_ROUTE_MAX_K) + " and at most the experts");
    if (r->normalize != 0 && r->normalize != 1)
        return fail(NS_EINVAL, "normalize must be 0 or 1");
    const size_t elt = dtype == NS_BF16 ? 2 : 4;
    if ((st = check_pointer("logits", r->logits, elt, r->tokens > 0)) != NS_OK ||
        (st = check_pointer("chosen", r->chosen, 4, r->tokens > 0)) != NS_OK)
        return st;
    if (r->ld < r->experts || r->ld > std::numeric_limits<int32_t>::max())
        return fail(NS_EINVAL, "the pitch of logits must be experts .. 2^31 - 1");
    return NS_OK;
}

// Parts of the workspace, from its start.
struct Parts {
    size_t probs, counts, routed, arrived, bytes;
};
Parts parts_of(int64_t groups, int64_t experts)
{
    Parts p{};
    if (groups == 1)
        return p;
    p.counts = (size_t)(groups * ((experts + kRouteJoin - 1) / kRouteJoin * kRouteJoin) * 4);
    p.routed = 2 * p.counts;
    p.arrived = p.routed + (size_t)groups * 4;
    p.bytes = p.arrived + 4;
    return p;
}

ns_status route(const ns_route* r, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    ns_status st;
    if ((st = check_common(r, dtype)) != NS_OK || (st = check_pointer("weights", r->weights, 4, r->tokens > 0)) != NS_OK ||
        (st = check_pointer("counts", r->counts, 4, true)) != NS_OK ||
        (st = check_pointer("probs", r->probs, 4, true)) != NS_OK ||
        (st = check_pointer("routed", r->routed, 4, true)) != NS_OK ||
        (st = check_pointer("loss", r->loss, 4, true)) != NS_OK)
        return st;
    const int64_t groups = route_groups(r->tokens, r->experts);
    const Parts p = parts_of(groups, r->experts);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes))
        return fail(NS_EINVAL, "a workspace of " + std::to_string(p.bytes) + " bytes is needed (ns_route_workspace_bytes)");
    if (p.bytes > 0 && reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(NS_EINVAL, "the workspace is not aligned to 16 bytes");
    char* ws = static_cast<char*>(workspace);
    RouteArgs a{};
    a.logits = static_cast<const char*>(r->logits);
    a.ld = r->ld;
    a.mask = r->mask;
    a.chosen = r->chosen;
    a.weights = r->weights;
    a.counts = r->counts;
    a.probs = r->probs;
    a.routed = r->routed;
    a.loss = r->loss;
    a.tokens = (int32_t)r->tokens;
    a.experts = (int32_t)r->experts;
    a.top_k = r->top_k;
    a.normalize = r->normalize;
    if (p.bytes > 0) {
        a.part_probs = reinterpret_cast<float*>(ws + p.probs);
        a.part_counts = reinterpret_cast<int32_t*>(ws + p.counts);
        a.part_routed = reinterpret_cast<int32_t*>(ws + p.routed);
        a.arrived = reinterpret_cast<uint32_t*>(ws + p.arrived);
    }
    st = launched(launch_route(a, (int)groups, dtype, stream), "router", stream);
    if (st == NS_OK && p.bytes > 0)
        st = launched(launch_route_join(a, (int)groups, stream), "router's sum", stream);
    return st;
}

ns_status route_grad(const ns_route_grad* g, int32_t dtype, hipStream_t stream)
{
    ns_status st;
    if ((st = check_common(g, dtype)) != NS_OK ||
        (st = check_pointer("counts", g->counts, 4, g->dloss != nullptr)) != NS_OK ||
        (st = check_pointer("routed", g->routed, 4, g->dloss != nullptr)) != NS_OK ||
        (st = check_pointer("dweights", g->dweights, 4, false)) != NS_OK ||
        (st = check_pointer("dloss", g->dloss, 4, false)) != NS_OK ||
        (st = check_pointer("out", g->out, dtype == NS_BF16 ? 2 : 4, g->tokens > 0)) != NS_OK)
        return st;
    if (g->ld_out < g->experts || g->ld_out > std::numeric_limits<int32_t>::max())
        return fail(NS_EINVAL, "the pitch of out must be experts .. 2^31 - 1");
    if (g->tokens == 0)
        return NS_OK;
    RouteGradArgs a{};
    a.logits = static_cast<const char*>(g->logits);
    a.ld = g->ld;
    a.chosen = g->chosen;
    a.counts = g->counts;
    a.routed = g->routed;
    a.dweights = g->dweights;
    a.dloss = g->dloss;
    a.out = static_cast<char*>(g->out);
    a.ldo = g->ld_out;
    a.tokens = (int32_t)g->tokens;
    a.experts = (int32_t)g->experts;
    a.top_k = g->top_k;
    a.normalize = g->normalize;
    const int64_t per = route_tokens(g->experts), groups = std::min<int64_t>((g->tokens + per - 1) / per, 2048);
    return launched(launch_route_grad(a, (int)groups, dtype, stream), "router's gradient", stream);
}

}  // namespace

extern "C" {

ns_status ns_route_experts(const ns_route* r, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&] { return route(r, dtype, workspace, workspace_bytes, static_cast<hipStream_t>(stream)); });
}

ns_status ns_route_workspace_bytes(int64_t tokens, int64_t experts, size_t* out_bytes)
{
    return guarded([&]() -> ns_status {
        if (!out_bytes)
            return fail(NS_EINVAL, "out_bytes must not be NULL");
        const ns_status st = check_sizes(tokens, experts);
        if (st == NS_OK)
            *out_bytes = parts_of(route_groups(tokens, experts), experts).bytes;
        return st;
    });
}

ns_status ns_route_experts_grad(const ns_route_grad* g, int32_t dtype, void* stream)
{
    return guarded([&] { return route_grad(g, dtype, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
