// Random attention plans over 4-bit pools on the CPU: every (cache head, row) of a sequence walks every key it sees once, the
// packs fit the kernel's columns and shared memory, the join's records cover every partial row once, and the counts stay
// within the capacities.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
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
    return j < kv_len && (full || j < prefix || (j <= p && (window == 0 || j > p - window)));
}

int main()
{
    std::mt19937_64 rng(11);
    auto below = [&](uint64_t n) { return (int64_t)(rng() % n); };
    // every shape of rows: the packs' pieces and their space in shared memory
    for (int groups = 1; groups <= 8; ++groups)
        for (int row = (17 * groups + 3) / 4 * 4; row < 17 * groups + 17; row += 4) {
            const int dp = groups <= 2 ? 64 : groups <= 4 ? 128 : 256, per = (row + 15) / 16;
            if (mx4_dim(row) != 32 * groups) continue;
            for (int heads = 1; heads <= 64; ++heads)
                for (int rows = 1; rows <= KVX_ROWS_FEW; ++rows)
                    for (int most = 1; most <= KVX_ROWS_FEW; most += 5) {
                        const int n = mx4_pack(heads, rows, row, dp, most);
                        CHECK(n >= 1 && heads % n == 0 && n * rows <= KVX_ROWS_FEW && (n <= most || n == 1));
                        CHECK(32 * n * per <= 64 * mx4_pieces(dp));
                        CHECK(n * 33 * per * 16 <= mx4_raw(dp));
                        CHECK(32 * n * per * 16 < 65536);  // divisions by a product
                    }
        }
    int64_t cut_pieces = 0, sizes[KVX_ROWS_FEW + 1] = {};
    for (int round = 0; round < 400; ++round) {
        const bool walk = round < 150;  // else counts alone, of more work
        kv_pool_desc d{};
        d.num_heads = below(2) ? 1 + (int32_t)below(9) : 4 << below(3);
        d.page_layout = below(3) ? KV_PAGE_TOKEN_MAJOR : KV_PAGE_HEAD_MAJOR;
        d.block_size = 16;
        const int32_t rows_of[] = {20, 36, 40, 48, 52, 68, 72, 80, 88, 104, 120, 136, 144};
        d.head_dim = rows_of[below(13)];
        kv_attn_desc a{};
        a.kv_type = KV_TYPE_MX4;
        a.num_q_heads = d.num_heads * (1 + (int32_t)below(9));
        const int mode = (int)below(4);
        a.window = mode == 1 || mode == 3 ? 1 + (int32_t)below(300) : 0;
        a.flags = mode == 2 ? KV_ATTN_FULL : 0;
        const int n = 1 + (int)below(walk ? 6 : 200);
        std::vector<kv_seq> seqs;
        int64_t at = 0;
        for (int i = 0; i < n; ++i) {
            kv_seq s{};
            s.block_table = (const int32_t *)(uintptr_t)(4096 * (i + 1));
            s.q_len = (int32_t)(below(3) ? below(4) : below(60));
            s.kv_len = below(5) ? s.q_len + below(500) : below(40);
            if (below(8) == 0) s.kv_len += walk ? 9000 : 90000;
            if (round % 20 == 0 && i == 0) s.kv_len = 180000, s.q_len = 1, s.prefix_len = 0;
            else s.prefix_len = below(2) ? 0 : (int32_t)below(700);
            s.q_begin = at;
            at += s.q_len;
            seqs.push_back(s);
        }
        a.max_seqs = n;
        a.max_tokens = at > 0 ? at : 1;
        const PlanLimits l = plan_limits(d, a);
        Plan p;
        p.reserve(l);
        const size_t held[3] = {p.few.capacity(), p.groups.capacity(), p.whole.capacity()};
        build_plan(p, l, seqs.data(), n);
        CHECK((int64_t)p.few.size() <= l.cap_few && (int64_t)p.many.size() <= l.cap_many);
        CHECK((int64_t)p.groups.size() <= l.cap_groups && (int64_t)p.append.size() <= l.cap_append);
        CHECK(p.few.capacity() == held[0] && p.groups.capacity() == held[1] && p.whole.capacity() == held[2]);
        std::map<std::tuple<const int32_t *, int, int64_t>, std::vector<uint8_t>> walked;
        std::map<int32_t, std::tuple<int32_t, int32_t, int32_t>> row_at;  // partial row -> (q_begin, head, row)
        std::map<std::tuple<int32_t, int32_t, int32_t>, int64_t> tiles;
        for (const AttnItem &it : p.few) {
            const int32_t rows = it.q_len * l.group;
            CHECK(it.row0 == 0 && rows >= 1 && it.across >= 1 && it.across * rows <= KVX_ROWS_FEW);
            CHECK(it.head >= 0 && it.head % it.across == 0 && it.head + it.across <= d.num_heads);
            ++sizes[it.across];
            const int32_t first = it.kv_len - it.q_len;
            const KeyWalk w = key_walk(it.kv_len, it.prefix, l.window, l.full, first, first + it.q_len - 1);
            CHECK(it.tile0 >= 0 && it.tile0 <= it.tile1 && it.tile1 <= w.n_tiles);
            if (it.prow >= 0) CHECK(it.prow + KVX_ROWS_FEW <= l.cap_prows);
            for (int h = 0; h < it.across; ++h)
                for (int32_t r = 0; r < rows; ++r) {
                    if (it.prow >= 0)
                        CHECK(row_at.emplace(it.prow + h * rows + r, std::make_tuple(it.q_begin, it.head + h, r)).second);
                    tiles[{it.q_begin, it.head + h, r}] += it.tile1 - it.tile0;
                    if (!walk) continue;
                    auto &keys = walked[{it.table, it.head + h, r}];
                    keys.resize((size_t)it.kv_len);
                    for (int32_t i = it.tile0; i < it.tile1; ++i)
                        for (int32_t j = w.start(i); j < w.start(i) + KVX_TILE_KEYS; ++j)
                            if (sees(it.kv_len, it.prefix, l.window, l.full, first + r / l.group, j)) ++keys[j];
                }
        }
        std::map<int32_t, int> joined;
        for (const AttnGroup &g : p.groups) {
            if ((int64_t)g.q_len * l.group > KVX_ROWS_FEW) continue;  // of the many-rows kernel
            ++cut_pieces;
            CHECK(g.rows >= 1 && g.rows <= KVX_JOIN_ROWS && g.n_parts >= 2);
            for (int k = 0; k < g.n_parts; ++k)
                for (int r = 0; r < g.rows; ++r) {
                    const auto f = row_at.find(g.prow + k * g.stride + r);
                    CHECK(f != row_at.end() && f->second == std::make_tuple(g.q_begin, g.head, g.row0 + r));
                    CHECK(++joined[f->first] == 1);
                }
        }
        CHECK(joined.size() == row_at.size());
        for (const kv_seq &s : seqs) {
            const int64_t rows = (int64_t)s.q_len * l.group;
            if (rows == 0 || rows > KVX_ROWS_FEW) continue;
            const int32_t first = (int32_t)(s.kv_len - s.q_len);
            const KeyWalk w = key_walk((int32_t)s.kv_len, s.prefix_len, l.window, l.full, first, first + s.q_len - 1);
            for (int h = 0; h < d.num_heads; ++h)
                for (int64_t r = 0; r < rows; ++r) {
                    const auto t = tiles.find({(int32_t)s.q_begin, h, (int32_t)r});
                    CHECK(t != tiles.end() && t->second == w.n_tiles);
                    if (!walk) continue;
                    const auto f = walked.find({s.block_table, h, r});
                    for (int64_t j = 0; j < s.kv_len; ++j)
                        CHECK(f->second[(size_t)j] ==
                              sees(s.kv_len, s.prefix_len, l.window, l.full, first + r / l.group, j));
                }
        }
    }
    CHECK(cut_pieces > 1000 && sizes[1] > 100 && sizes[2] > 100 && sizes[4] > 100);
    std::printf("ok\n");
    return 0;
}
