// The split search of attention plans on the CPU: the span of parts that are counted together is that of parts dealt one by one,
// and sequences of unequal packs (4-bit pools, single tokens beside drafts) take it no more runs than two for each.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <queue>
#include <random>

#include "kvxfer_plan.h"

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("failed: %s (line %d)\n", #x, __LINE__);      \
            std::exit(1);                                             \
        }                                                             \
    } while (0)

using namespace kvx;

// Every part of every pack dealt to the workgroup that ends first.
static int64_t dealt(const std::vector<AttnItem> &whole, int64_t share, int64_t slots, const SplitCost &cost, Weight weight)
{
    std::vector<int64_t> parts;
    bool any = false;
    for (const AttnItem &it : whole) {
        const int64_t n = std::max<int64_t>(1, (it.tile1 + share - 1) / share);
        any |= n > 1;
        for (int64_t w = 0; w < weight(it); ++w)
            for (int64_t k = 0; k < n; ++k)
                parts.push_back(it.tile1 * (k + 1) / n - it.tile1 * k / n + (n > 1 ? cost.cut : cost.whole));
    }
    std::sort(parts.rbegin(), parts.rend());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
    for (int64_t i = 0; i < slots; ++i) ends.push(0);
    int64_t last = 0;
    for (const int64_t p : parts) {
        const int64_t end = ends.top() + p;
        ends.pop();
        ends.push(end);
        last = std::max(last, end);
    }
    return last + (any ? cost.join : 0);
}

int main()
{
    std::mt19937_64 rng(3);
    auto below = [&](uint64_t n) { return (int64_t)(rng() % n); };
    std::vector<int64_t> parts, ends;
    for (int round = 0; round < 2000; ++round) {
        const int32_t heads = 1 << below(5);
        std::vector<AttnItem> whole((size_t)(1 + below(40)));
        const bool weighed = below(2), few = below(2);
        for (AttnItem &it : whole) {
            it.tile1 = (int32_t)(below(4) ? below(12) : below(3000));
            it.across = (int16_t)(1 << below(4));
            while (it.across > heads) it.across /= 2;
        }
        const Weight weight{weighed ? heads : 0};
        const int64_t share = 1 + below(200), slots = 1 + below(512);
        const SplitCost &cost = few ? kCostFew : kCostMany;
        CHECK(span_at(whole, share, slots, cost, weight, parts, ends) == dealt(whole, share, slots, cost, weight));
        int64_t n = 0;
        for (const AttnItem &it : whole) n += std::max<int64_t>(1, (it.tile1 + share - 1) / share) * weight(it) * 3;
        CHECK(parts_at(whole, share, 3, weight) == n);
    }
    for (int n : {3, 16, 64, 128, 256}) {
        kv_pool_desc d{};
        d.num_heads = 8;
        d.block_size = 16;
        d.head_dim = 68;
        d.elem_bytes = 1;
        kv_attn_desc a{};
        a.kv_type = KV_TYPE_MX4;
        a.num_q_heads = 32;
        a.max_seqs = n;
        std::vector<kv_seq> seqs((size_t)n);
        for (int i = 0; i < n; ++i) {
            seqs[i] = kv_seq{};
            seqs[i].block_table = (const int32_t *)(uintptr_t)4096;
            seqs[i].q_len = i % 2 ? 4 : 1;
            seqs[i].kv_len = 1024 + below(31000);
            seqs[i].q_begin = a.max_tokens;
            a.max_tokens += seqs[i].q_len;
        }
        const PlanLimits l = plan_limits(d, a);
        Plan p;
        p.reserve(l);
        const size_t held[2] = {p.parts.capacity(), p.ends.capacity()};
        build_plan(p, l, seqs.data(), n);
        CHECK(!p.few.empty() && p.parts.size() <= 2 * (size_t)n);
        CHECK(p.parts.capacity() == held[0] && p.ends.capacity() == held[1]);
    }
    std::puts("ok");
}
