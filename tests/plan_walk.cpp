// Random attention plans on the CPU: every (row, visible key) pair of a plan is walked by
// exactly one piece, no piece walks a tile no row of it sees, the pieces of a group are what
// the join reads, and the counts stay within the capacities.  Also division by
// multiplication.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>

#include "kvxfer_plan.h"

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("failed: %s (line %d)\n", #x, __LINE__);      \
            std::exit(1);                                             \
        }                                                             \
    } while (0)

using namespace kvx;

static bool sees(int64_t kv_len, int64_t prefix, int64_t window, bool full, int64_t p, int64_t j)
{
    if (j >= kv_len) return false;
    return full || j < prefix || (j <= p && (window == 0 || j > p - window));
}

int main()
{
    std::mt19937_64 rng(7);
    auto below = [&](uint64_t n) { return (int64_t)(rng() % n); };
    for (uint32_t d : {1u, 2u, 3u, 5u, 7u, 16u, 24u, 48u, 100u, 255u, 256u, 65537u, 0x7fffffffu}) {
        uint32_t m, s;
        set_div(d, &m, &s);
        for (int i = 0; i < 20000; ++i) {
            const uint32_t x = i < 10 ? (uint32_t)(0x7fffffff - i) : (uint32_t)below(0x80000000ull);
            CHECK(div_by(x, m, s) == x / d);
            const uint32_t y = x / d * d;
            CHECK(div_by(y, m, s) == y / d);
            if (y) CHECK(div_by(y - 1, m, s) == (y - 1) / d);
        }
    }
    for (int round = 0; round < 120; ++round) {
        kv_pool_desc d{};
        d.num_heads = below(3) ? 1 + (int32_t)below(3) : 4;
        d.page_layout = below(3) ? KV_PAGE_TOKEN_MAJOR : KV_PAGE_HEAD_MAJOR;
        d.block_size = 16;
        kv_attn_desc a{};
        d.head_dim = below(2) ? 64 : 256;
        a.num_q_heads = d.num_heads * (1 + (int32_t)below(9));
        const int mode = (int)below(4);
        a.window = mode == 1 || mode == 3 ? (below(6) ? 1 + (int32_t)below(300) : INT32_MAX - (int32_t)below(3)) : 0;
        a.flags = mode == 2 ? KV_ATTN_FULL : 0;
        const int n = 1 + (int)below(6);
        std::vector<kv_seq> seqs;
        int64_t at = 0;
        for (int i = 0; i < n; ++i) {
            kv_seq s{};
            s.block_table = (const int32_t *)(uintptr_t)(4096 * (i + 1));
            s.q_len = (int32_t)(below(3) ? below(4) : below(60));
            s.kv_len = below(5) ? s.q_len + below(500) : below(40);  // some shorter than their queries
            if (below(8) == 0) s.kv_len += 9000;
            if (round % 20 == 0 && i == 0) s.kv_len = 180000, s.q_len = 1, s.prefix_len = 0;  // work for a head a wave
            s.prefix_len = below(2) ? 0 : (int32_t)below(700);
            s.q_begin = at;
            at += s.q_len;
            seqs.push_back(s);
        }
        a.max_seqs = n;
        a.max_tokens = at > 0 ? at : 1;
        const PlanLimits l = plan_limits(d, a);
        Plan p;
        build_plan(p, l, seqs.data(), n);
        CHECK((int64_t)p.few.size() <= l.cap_few && (int64_t)p.many.size() <= l.cap_many);
        CHECK((int64_t)p.groups.size() <= l.cap_groups && (int64_t)p.append.size() <= l.cap_append);
        CHECK(p.tokens_end == at);
        std::map<std::tuple<const int32_t *, int, int64_t>, std::vector<uint8_t>> walked;
        std::map<int32_t, std::tuple<int32_t, int32_t, int32_t>> parts;  // prow -> (q_begin, head, row0)
        for (int cls = 0; cls < 2; ++cls)
            for (const AttnItem &whole : cls ? p.many : p.few)
            for (int wave = 0; wave < (whole.across ? 4 : 1); ++wave) {  // a head to each wave
                AttnItem it = whole;
                CHECK(!whole.across || !cls);
                it.head += wave;
                if (it.prow >= 0) it.prow += 16 * wave;
                const int step = it.rows;
                CHECK(step == (cls ? l.rows_many : KVX_ROWS_FEW) || (cls && step == KVX_ROWS_HALF));
                CHECK(it.head >= 0 && it.head < d.num_heads && it.row0 % step == 0);
                const int64_t rows = std::min<int64_t>(step, (int64_t)it.q_len * l.group - it.row0);
                CHECK(rows > 0);
                const int32_t first = it.kv_len - it.q_len;
                const KeyWalk w = key_walk(it.kv_len, it.prefix, l.window, l.full, first + it.row0 / l.group,
                                           first + (int32_t)((it.row0 + rows - 1) / l.group));
                CHECK(it.tile0 >= 0 && it.tile0 <= it.tile1 && it.tile1 <= w.n_tiles);
                if (it.prow >= 0) {
                    CHECK(it.prow % KVX_ROWS_FEW == 0 && it.prow + step <= l.cap_prows);
                    CHECK(parts.emplace(it.prow, std::make_tuple(it.q_begin, it.head, it.row0)).second);
                }
                for (int64_t r = it.row0; r < it.row0 + rows; ++r) {
                    auto &keys = walked[{it.table, it.head, r}];
                    keys.resize((size_t)it.kv_len);
                    const int64_t pos = first + r / l.group;
                    for (int32_t i = it.tile0; i < it.tile1; ++i) {
                        const int32_t j0 = w.start(i);
                        CHECK(j0 >= 0 && j0 < it.kv_len);
                        for (int32_t j = j0; j < j0 + KVX_TILE_KEYS; ++j) {
                            const bool any = j < w.prefix || (j >= w.low && j < w.high);
                            if (sees(it.kv_len, it.prefix, l.window, l.full, pos, j)) {
                                CHECK(any);
                                ++keys[j];
                            }
                            if (any) CHECK(j < it.kv_len);
                        }
                    }
                }
            }
        std::map<int32_t, int32_t> joined;  // prow of a part -> its rows that some record joins
        for (const AttnGroup &g : p.groups)
            for (int k = 0; k < g.n_parts; ++k) {
                // a record starts at some row of the part
                auto f = parts.upper_bound(g.prow + k * g.stride);
                CHECK(f != parts.begin());
                --f;
                const int32_t off = g.prow + k * g.stride - f->first;
                CHECK(off >= 0 && off + g.rows <= g.stride && g.rows >= 1 && g.rows <= KVX_JOIN_ROWS);
                CHECK(f->second == std::make_tuple(g.q_begin, g.head, g.row0 - off));
                CHECK(joined[f->first] == off);
                joined[f->first] += g.rows;
            }
        for (int cls = 0; cls < 2; ++cls)
            for (const AttnItem &it : cls ? p.many : p.few)
                for (int wave = 0; it.prow >= 0 && wave < (it.across ? 4 : 1); ++wave) {
                    const int64_t rows = std::min<int64_t>(it.rows,
                                                           (int64_t)it.q_len * l.group - it.row0);
                    CHECK(joined[it.prow + 16 * wave] == rows);
                }
        CHECK(joined.size() == parts.size());
        std::set<std::pair<const int32_t *, int>> appended;
        for (const AppendItem &it : p.append)
            for (int k = 0; k < it.count; ++k) CHECK(appended.emplace(it.table, it.pos + k).second);
        size_t news = 0;
        for (const kv_seq &s : seqs) {
            if (s.q_len <= s.kv_len) news += s.q_len;
            for (int h = 0; h < d.num_heads; ++h)
                for (int64_t r = 0; r < (int64_t)s.q_len * l.group; ++r) {
                    const auto f = walked.find({s.block_table, h, r});
                    CHECK(f != walked.end());
                    for (int64_t j = 0; j < s.kv_len; ++j)
                        CHECK(f->second[(size_t)j] ==
                              sees(s.kv_len, s.prefix_len, l.window, l.full, s.kv_len - s.q_len + r / l.group, j));
                }
        }
        CHECK(appended.size() == (p.appendable ? news : 0));
    }
    // counts alone, of larger steps: half pieces and whole ones, cut and uncut
    int halves = 0, wholes = 0, cuts = 0;
    for (int round = 0; round < 1500; ++round) {
        kv_pool_desc d{};
        d.num_heads = 1 + (int32_t)below(8);
        d.page_layout = KV_PAGE_TOKEN_MAJOR;
        d.block_size = 16;
        kv_attn_desc a{};
        d.head_dim = below(4) ? 128 : 256;
        a.num_q_heads = d.num_heads * (1 + (int32_t)below(8));
        a.window = below(4) ? 0 : 1 + (int32_t)below(5000);
        std::vector<kv_seq> seqs;
        int64_t at = 0;
        const int n = 1 + (int)below(below(2) ? 3 : 40);
        for (int i = 0; i < n; ++i) {
            kv_seq s{};
            s.block_table = (const int32_t *)(uintptr_t)4096;
            s.q_len = (int32_t)(below(3) ? 1 + below(1 << below(13)) : 1);
            s.kv_len = s.q_len + (below(2) ? below(1 << below(18)) : 0);
            s.q_begin = at;
            at += s.q_len;
            seqs.push_back(s);
        }
        a.max_seqs = n;
        a.max_tokens = at;
        const PlanLimits l = plan_limits(d, a);
        Plan p;
        build_plan(p, l, seqs.data(), n);
        CHECK((int64_t)p.few.size() <= l.cap_few && (int64_t)p.many.size() <= l.cap_many);
        CHECK((int64_t)p.groups.size() <= l.cap_groups && (int64_t)p.append.size() <= l.cap_append);
        int64_t rows = 0, want = 0;
        for (int cls = 0; cls < 2; ++cls)
            for (const AttnItem &it : cls ? p.many : p.few) {
                const int64_t r = std::min<int64_t>(it.rows, (int64_t)it.q_len * l.group - it.row0);
                if (it.prow >= 0) CHECK(it.prow + (int64_t)it.rows * (it.across ? 4 : 1) <= l.cap_prows);
                if (it.tile0 == 0) rows += r * (it.across ? 4 : 1);
                if (cls) halves += it.rows < l.rows_many, wholes += it.rows == l.rows_many, cuts += it.prow >= 0;
            }
        for (const kv_seq &s : seqs) want += (int64_t)s.q_len * l.group * d.num_heads;
        CHECK(rows == want);
    }
    CHECK(halves > 1000 && wholes > 1000 && cuts > 1000);
    std::printf("ok\n");
    return 0;
}
