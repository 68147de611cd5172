// q8_workspace.cu -- which words of the callers' workspaces are known to be zero.
//
// The words that kernels count with (split-K tickets, the GEMV's pool counter,
// the attention's tickets, the experts' arrivals) are zero before every launch
// and left zero by it, but where they lie depends on the call and its shapes,
// and calls may share a workspace in stream order: one call's partial sums, x
// copies or hidden units may lie where the next call counts.  So the library
// keeps the ranges of device addresses that a call counted with (zero since) and
// no later call wrote data to.  A call clears those of its counters that are not
// among them, one memset each in its stream: on the first use of an address,
// and after a call that wrote there.  Calls that repeat the same shapes clear
// nothing.  Addresses, not workspaces: a chain's regions, a part of a workspace
// and the whole of it are seen as what they are.
#include <iterator>
#include <map>
#include <mutex>
#include <new>

#include "q8_internal.h"

namespace q8 {

namespace {

std::mutex g_mu;
std::map<uintptr_t, uintptr_t> g_zero;  // disjoint [first, second), no two of them adjacent
constexpr size_t kMaxRanges = 1 << 16;  // beyond that all are forgotten (and cleared on their next use)

bool known_zero(uintptr_t a, uintptr_t b) {
    auto it = g_zero.upper_bound(a);
    return it != g_zero.begin() && std::prev(it)->second >= b;
}

void forget(uintptr_t a, uintptr_t b) {
    auto it = g_zero.upper_bound(a);
    if (it != g_zero.begin() && std::prev(it)->second > a) --it;
    while (it != g_zero.end() && it->first < b) {
        const uintptr_t first = it->first, second = it->second;
        it = g_zero.erase(it);
        if (first < a) g_zero.emplace(first, a);
        if (second > b) g_zero.emplace(b, second);
    }
}

void remember(uintptr_t a, uintptr_t b) {
    if (known_zero(a, b)) return;
    forget(a, b);
    auto it = g_zero.lower_bound(a);
    if (it != g_zero.end() && it->first == b) {
        b = it->second;
        it = g_zero.erase(it);
    }
    if (it != g_zero.begin() && std::prev(it)->second == a)
        std::prev(it)->second = b;
    else
        g_zero.emplace(a, b);
}

}  // namespace

q8_status claim_workspace(void *ws, const WsRange *counters, size_t ncounters, const WsRange *data, size_t ndata,
                          cudaStream_t stream) {
    if (ws == nullptr) return Q8_OK;
    const uintptr_t base = reinterpret_cast<uintptr_t>(ws);
    std::lock_guard<std::mutex> lock(g_mu);
    for (size_t i = 0; i < ncounters; ++i) {
        const WsRange &r = counters[i];
        if (known_zero(base + r.off, base + r.off + r.len)) continue;
        if (cudaMemsetAsync(static_cast<uint8_t *>(ws) + r.off, 0, r.len, stream) != cudaSuccess) return Q8_ERR_CUDA;
    }
    try {
        for (size_t i = 0; i < ncounters; ++i) remember(base + counters[i].off, base + counters[i].off + counters[i].len);
        for (size_t i = 0; i < ndata; ++i) forget(base + data[i].off, base + data[i].off + data[i].len);
        if (g_zero.size() > kMaxRanges) g_zero.clear();
    } catch (const std::bad_alloc &) {
        g_zero.clear();  // nothing is known: cleared on its next use
    }
    return Q8_OK;
}

}  // namespace q8
