// kvxfer_plan.h -- host planning of one step's attention: which pieces of work there are
// and how they are split over the keys (host only; no HIP call; the vectors keep their
// capacity, and std::stable_sort takes a buffer for the call).  On a host of the measured card a set takes 6 us for one
// short decode, 9 for one on 32 K tokens, 17 for 16 sequences, 26 for 64 or for eight ragged turns, 53 for 256,
// its upload's call included.
#pragma once
#include <algorithm>
#include <functional>
#include <vector>

#include "kvxfer_ops.h"

namespace kvx {

// Workgroups that run at once: two to a compute unit for few rows (four waves of at most 256
// registers; one for the widest heads), one of up to eight waves for many rows.
inline int32_t slots_few(int dim) { return dim > 128 ? 256 : 512; }
constexpr int32_t kSlotsMany = 256;

struct PlanLimits {
    int32_t heads, group, window, rows_many, slots_few;
    bool full, token_major;
    int64_t cap_few, cap_many, cap_groups, cap_append, cap_prows;
};

// Capacities that hold any plan of max_seqs sequences and max_tokens new tokens.  Of a class
// with at most `pieces` pieces, at most cut_parts() parts are cut, and at most all_parts()
// made in all.
inline int64_t max_rounds(int64_t pieces, int64_t slots) { return pieces <= slots ? 2 : 4; }
inline int64_t cut_parts(int64_t pieces, int64_t slots) { return max_rounds(pieces, slots) * slots; }
inline int64_t all_parts(int64_t pieces, int64_t slots)
{
    return std::max(cut_parts(pieces, slots), pieces >= 4 * slots ? pieces + 2 * slots : 0);
}

inline PlanLimits plan_limits(const kv_pool_desc &d, const kv_attn_desc &a)
{
    PlanLimits l;
    l.heads = d.num_heads;
    l.group = a.num_q_heads / d.num_heads;
    l.window = a.window;
    l.full = (a.flags & KV_ATTN_FULL) != 0;
    l.token_major = d.page_layout == KV_PAGE_TOKEN_MAJOR;
    l.rows_many = rows_many(d.head_dim);
    l.slots_few = slots_few(d.head_dim);
    const int64_t rows = a.max_tokens * l.group;
    const int64_t seqs = std::min<int64_t>(a.max_seqs, a.max_tokens);
    auto slices = [](int64_t n) { return (n + KVX_JOIN_ROWS - 1) / KVX_JOIN_ROWS; };
    const int64_t few = seqs * l.heads, cut_few = cut_parts(few, l.slots_few);
    l.cap_few = all_parts(few, l.slots_few);
    // a cut piece has two parts or more, and one record for KVX_JOIN_ROWS of its rows
    const int64_t heads_cut = l.heads % 4 == 0 ? 4 : 1;  // of one piece (Split::across)
    l.cap_groups = std::min(cut_few / 2 * heads_cut, few) * slices(std::min<int64_t>(rows, KVX_ROWS_FEW));
    l.cap_prows = cut_few * KVX_ROWS_FEW * heads_cut;
    l.cap_many = 0;
    if (rows > KVX_ROWS_FEW) {
        const int64_t many = (rows / l.rows_many + seqs) * l.heads, cut_many = cut_parts(many, kSlotsMany);
        l.cap_many = all_parts(many, kSlotsMany);
        l.cap_groups += std::min(cut_many / 2, many) * slices(std::min<int64_t>(rows, l.rows_many));
        l.cap_prows += cut_many * l.rows_many;
    }
    l.cap_append = a.max_tokens / KVX_APPEND_TOKENS + seqs;
    return l;
}

struct Plan {
    PlanHead head{};
    std::vector<AttnItem> few, many;
    std::vector<AttnGroup> groups;
    std::vector<AppendItem> append;
    int64_t tokens_end = 0;   // one past the last row any sequence owns
    bool appendable = true;   // every sequence has q_len <= kv_len
    // scratch
    std::vector<AttnItem> whole;
    std::vector<int64_t> parts, ends;

    void reserve(const PlanLimits &l)
    {
        few.reserve(l.cap_few);
        many.reserve(l.cap_many);
        whole.reserve(std::max(l.cap_few, l.cap_many));
        groups.reserve(l.cap_groups);
        append.reserve(l.cap_append);
        parts.reserve(8 * (size_t)std::max(l.slots_few, kSlotsMany));
        ends.reserve((size_t)std::max(l.slots_few, kSlotsMany));
    }
};

// Parts that `share` tiles at most cut the pieces into, all cache heads together.
inline int64_t parts_at(const std::vector<AttnItem> &whole, int64_t share, int32_t heads)
{
    int64_t n = 0;
    for (const AttnItem &it : whole) n += std::max<int64_t>(1, (it.tile1 + share - 1) / share);
    return n * heads;
}

// What splitting costs, in the time of one tile: a part's start and end, whole or cut, and the join.
// Many rows: a cut part writes up to 128 KiB that the join reads, a tile's time or two each way at a compute
// unit's share of HBM (ragged 64-wide turns: 90 us at a cost of 2 or 4, 110 us at 6, where too
// little is cut); the join's launch two to four (with 2 prompts of 1024 and 1536 tokens were cut,
// 38.7 and 50 us, and now are not).  Few rows: a part's 8 KiB are nothing, but the join's 4 us are ten
// tiles of a workgroup.
struct SplitCost {
    int64_t whole, cut, join, min_tiles;
};
// Measured in tiles of 128-wide 16-bit heads without a cap, and used for all: a 64-wide tile costs less, a capped
// one more, and with them the costs in tiles.
constexpr SplitCost kCostFew{2, 2, 10, 2}, kCostMany{1, 4, 4, 8}, kCostHalf{1, 4, 5, 8};
// A tile with waves 0 to 3 at work takes 72 hundredths of the time of one with all (1.5 and
// 2.1 us, 128-wide heads; 512 new tokens on 16 K cached, cut to one round either way: 217 and 155 us).
constexpr int64_t kHalfTile = 72;

// When the last of `slots` workgroups ends, in tiles, if each takes the longest part left.
// `ends` is scratch.
inline int64_t span_at(const std::vector<AttnItem> &whole, int64_t share, int64_t slots, const SplitCost &cost,
                       std::vector<int64_t> &parts, std::vector<int64_t> &ends)
{
    parts.clear();
    bool any = false;
    for (const AttnItem &it : whole) {
        const int64_t n = std::max<int64_t>(1, (it.tile1 + share - 1) / share);
        any |= n > 1;
        for (int64_t k = 0; k < n; ++k)
            parts.push_back(it.tile1 * (k + 1) / n - it.tile1 * k / n + (n > 1 ? cost.cut : cost.whole));
    }
    std::sort(parts.begin(), parts.end(), std::greater<int64_t>());
    ends.assign((size_t)slots, 0);  // a heap, the earliest end first
    for (int64_t p : parts) {
        std::pop_heap(ends.begin(), ends.end(), std::greater<int64_t>());
        ends.back() += p;
        std::push_heap(ends.begin(), ends.end(), std::greater<int64_t>());
    }
    return *std::max_element(ends.begin(), ends.end()) + (any ? cost.join : 0);
}

// Splits the pieces in `whole` (tile0 = 0, tile1 = all tiles, one for all cache heads) over the keys.
//  * At least four times as many pieces as workgroups that run at once (slots): only pieces longer
//    than the even share are cut; the rest even out by themselves, longest first.  A piece of t >
//    share tiles gives at most t / share + 1 < 2 t / share parts, and the sum of t / share is at
//    most slots.
//  * Fewer: no cut, the smallest share whose parts fill one, two, ... rounds, or the longest piece
//    cut in two, three or four and the others where they are longer, whichever ends first.  One
//    round suits equal pieces; more even out unequal ones (32 sequences of 1 K to 64 K tokens: one
//    round 353 us, two 335 us, four 333 us; one sequence of 32 K: 34, 38, 49 us).
// Without the costs of a cut, a prompt of 2048 tokens was cut into parts of 11 tiles and took 68 us.
struct Split {
    int64_t share, span;  // tiles of a part at most; when the last workgroup ends, in tiles (0: not asked)
    int32_t across;       // cache heads of a workgroup
};
inline Split choose_split(Plan &p, const PlanLimits &l, int64_t slots, const SplitCost &cost, bool few,
                          int64_t parts_max = INT64_MAX)
{
    int64_t total = 0, longest = 1;
    for (const AttnItem &it : p.whole)
        total += (int64_t)it.tile1 * l.heads, longest = std::max<int64_t>(longest, it.tile1);
    // Four heads to a workgroup where they are neighbours in a page and there is work enough to
    // give every wave some steps of its head.
    const int32_t across = few && l.token_major && l.heads % 4 == 0 && total >= KVX_ACROSS * slots ? 4 : 1;
    const int32_t units = l.heads / across;
    total /= across;
    const int64_t even = std::max(cost.min_tiles, (total + slots - 1) / slots);
    const int64_t pieces = (int64_t)p.whole.size() * units;
    parts_max = std::min(parts_max, cut_parts(pieces, slots));
    auto fitting = [&](int64_t parts) {
        int64_t lo = std::min(cost.min_tiles, longest), hi = longest;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (parts_at(p.whole, mid, units) <= parts) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    Split out{longest, 0, across};
    if (pieces >= 4 * slots) {
        out.share = std::min(even, longest);
    } else {
        const int64_t lanes = std::max<int64_t>(1, slots / units);
        const int64_t uncut = span_at(p.whole, longest, lanes, cost, p.parts, p.ends);
        out.span = uncut;
        int64_t best = (uncut * 19 + 19) / 20;  // a cut for less than a twentieth is not worth its risk
        auto consider = [&](int64_t s) {
            if (s >= longest || parts_at(p.whole, s, units) > parts_max) return;
            const int64_t span = span_at(p.whole, s, lanes, cost, p.parts, p.ends);
            if (span < best) out.span = best = span, out.share = s;
        };
        for (int64_t rounds = 1; rounds * slots <= parts_max; ++rounds)
            if (pieces <= rounds * slots) consider(fitting(rounds * slots));
        for (int64_t cuts = 2; cuts <= 4; ++cuts) consider(std::max(cost.min_tiles, (longest + cuts - 1) / cuts));
    }
    return out;
}

// The parts of the pieces in `whole`, longest first, and the records that join them.
inline void cut(Plan &p, std::vector<AttnItem> &out, const PlanLimits &l, int32_t rows_of_piece, const Split &split,
                int64_t *prow)
{
    const int64_t share = split.share;
    const int32_t across = split.across, units = l.heads / across;
    for (const AttnItem &it : p.whole) {
        const int64_t n = (it.tile1 + share - 1) / share;
        const int32_t rows = (int32_t)std::min<int64_t>(rows_of_piece, (int64_t)it.q_len * l.group - it.row0);
        AttnItem part = it;
        part.across = across > 1;
        if (n <= 1) {
            for (part.head = 0; part.head < l.heads; part.head += across) out.push_back(part);
            continue;
        }
        // part k of head h at prow + (h / across * n + k) * stride + h mod across * 16
        const int32_t stride = rows_of_piece * across;
        for (int32_t head = 0; head < l.heads; ++head)
            for (int32_t r = 0; r < rows; r += KVX_JOIN_ROWS)
                p.groups.push_back(AttnGroup{
                    (int32_t)(*prow + head / across * n * stride + head % across * rows_of_piece + r), (int32_t)n,
                    stride, std::min(KVX_JOIN_ROWS, rows - r), it.q_begin, it.q_len, head, it.row0 + r});
        // the heads of one stretch of keys side by side: they read neighbouring bytes of one page
        for (int64_t k = 0; k < n; ++k)
            for (int32_t head = 0; head < l.heads; head += across) {
                part.head = head;
                part.tile0 = (int32_t)(it.tile1 * k / n);
                part.tile1 = (int32_t)(it.tile1 * (k + 1) / n);
                part.prow = (int32_t)(*prow + (head / across * n + k) * stride);
                out.push_back(part);
            }
        *prow += units * n * stride;
    }
    // longest first, so that the last workgroups to start are the short ones
    std::stable_sort(out.begin(), out.end(), [](const AttnItem &a, const AttnItem &b) {
        return a.tile1 - a.tile0 > b.tile1 - b.tile0;
    });
}

// The pieces of the few rows' or the many rows' sequences into `whole`, `step` rows each; the largest's rows.
inline int32_t pieces_of(Plan &p, const PlanLimits &l, const kv_seq *seqs, int32_t n, bool few, int32_t step)
{
    int32_t most = 0;
    p.whole.clear();
    for (int32_t i = 0; i < n; ++i) {
        const kv_seq &s = seqs[i];
        const int64_t rows = (int64_t)s.q_len * l.group;
        if (rows == 0 || (rows <= KVX_ROWS_FEW) != few) continue;
        most = std::max(most, (int32_t)std::min<int64_t>(rows, step));
        for (int64_t r = 0; r < rows; r += step) {
            const int32_t t0 = (int32_t)(r / l.group);
            const int32_t t1 = (int32_t)((std::min(rows, r + step) - 1) / l.group);
            const int32_t first = (int32_t)(s.kv_len - s.q_len);
            const KeyWalk w = key_walk((int32_t)s.kv_len, s.prefix_len, l.window, l.full, first + t0, first + t1);
            AttnItem it{};
            it.table = s.block_table;
            it.kv_len = (int32_t)s.kv_len;
            it.q_begin = (int32_t)s.q_begin;
            it.q_len = s.q_len;
            it.prefix = s.prefix_len;
            it.row0 = (int32_t)r;
            it.tile1 = w.n_tiles;
            it.prow = -1;
            it.rows = (int16_t)step;
            p.whole.push_back(it);
        }
    }
    return most;
}

// The plan of checked sequences.
inline void build_plan(Plan &p, const PlanLimits &l, const kv_seq *seqs, int32_t n)
{
    p.few.clear();
    p.many.clear();
    p.groups.clear();
    p.append.clear();
    p.tokens_end = 0;
    p.appendable = true;
    int64_t prow = 0;
    if (pieces_of(p, l, seqs, n, true, KVX_ROWS_FEW) > 0)
        cut(p, p.few, l, KVX_ROWS_FEW, choose_split(p, l, l.slots_few, kCostFew, true), &prow);
    int32_t step = l.rows_many;
    if (const int32_t rows = pieces_of(p, l, seqs, n, false, step)) {
        Split split = choose_split(p, l, kSlotsMany, kCostMany, false);
        // Half the rows in twice as many pieces, at most two to a workgroup that runs at once, for steps
        // that do not fill the chip otherwise.  128-wide heads, 32 on 8: a prompt of 256 tokens 17.4 -> 13.8
        // us, of 1024 38.6 -> 31.7, of 2048 67.7 -> 65.3; 1024 new on 5000 through a window of 1000 43 -> 36;
        // worst seen, six ragged sequences of 40 to 1500 new tokens, 52 -> 56.
        if (rows > KVX_ROWS_HALF && split.span) {
            pieces_of(p, l, seqs, n, false, KVX_ROWS_HALF);
            if ((int64_t)p.whole.size() * l.heads <= 2 * kSlotsMany) {
                const Split half = choose_split(p, l, kSlotsMany, kCostHalf, false, 2 * kSlotsMany);
                if (half.span * kHalfTile < split.span * 100) split = half, step = KVX_ROWS_HALF;
            }
            if (step != KVX_ROWS_HALF) pieces_of(p, l, seqs, n, false, step);
        }
        cut(p, p.many, l, step, split, &prow);
    }
    for (int32_t i = 0; i < n; ++i) {
        const kv_seq &s = seqs[i];
        if (s.q_len == 0) continue;
        p.tokens_end = std::max<int64_t>(p.tokens_end, s.q_begin + s.q_len);
        if (s.q_len > s.kv_len) p.appendable = false;
        for (int32_t t = 0; t < s.q_len; t += KVX_APPEND_TOKENS)
            p.append.push_back(AppendItem{s.block_table, (int32_t)(s.kv_len - s.q_len) + t, (int32_t)s.q_begin + t,
                                          std::min(KVX_APPEND_TOKENS, s.q_len - t), 0});
    }
    if (!p.appendable) p.append.clear();  // a replay of a captured append then writes nothing
    p.head.n_few = (int32_t)p.few.size();
    p.head.n_many = (int32_t)p.many.size();
    p.head.n_groups = (int32_t)p.groups.size();
    p.head.n_append = (int32_t)p.append.size();
}

}  // namespace kvx
