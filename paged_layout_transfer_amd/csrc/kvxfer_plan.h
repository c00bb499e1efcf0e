// kvxfer_plan.h -- host planning of one step's attention: which pieces of work there are
// and how they are split over the keys (host only; no HIP call, no allocation once the
// vectors have their capacity).
#pragma once
#include <algorithm>
#include <vector>

#include "kvxfer_ops.h"

namespace kvx {

// Workgroups that run at once: two to a compute unit for few rows (four waves of at most 256
// registers; one for the widest heads), one of up to eight waves for many rows.
inline int32_t slots_few(int dim) { return dim > 128 ? 256 : 512; }
constexpr int32_t kSlotsMany = 256;

struct PlanLimits {
    int32_t heads, group, window, rows_many, slots_few;
    bool full;
    int64_t cap_few, cap_many, cap_groups, cap_append, cap_prows;
};

// Capacities that hold any plan of max_seqs sequences and max_tokens new tokens.  Splitting
// makes at most 2 * slots pieces of a class (split_class), each with its rows in the workspace.
inline PlanLimits plan_limits(const kv_pool_desc &d, const kv_attn_desc &a)
{
    PlanLimits l;
    l.heads = d.num_heads;
    l.group = a.num_q_heads / d.num_heads;
    l.window = a.window;
    l.full = (a.flags & KV_ATTN_FULL) != 0;
    l.rows_many = rows_many(d.head_dim);
    l.slots_few = slots_few(d.head_dim);
    const int64_t rows = a.max_tokens * l.group;
    const int64_t seqs = std::min<int64_t>(a.max_seqs, a.max_tokens);
    const bool many = rows > KVX_ROWS_FEW;
    l.cap_few = seqs * l.heads + 2 * l.slots_few;
    l.cap_many = many ? (rows / l.rows_many + seqs) * l.heads + 2 * kSlotsMany : 0;
    const int64_t few_rows = std::min<int64_t>(rows, KVX_ROWS_FEW), many_rows = std::min<int64_t>(rows, l.rows_many);
    l.cap_groups = l.slots_few * ((few_rows + KVX_JOIN_ROWS - 1) / KVX_JOIN_ROWS) +
                   (many ? kSlotsMany * ((many_rows + KVX_JOIN_ROWS - 1) / KVX_JOIN_ROWS) : 0);
    l.cap_append = a.max_tokens / KVX_APPEND_TOKENS + seqs;
    l.cap_prows = 2 * l.slots_few * KVX_ROWS_FEW + (many ? 2 * kSlotsMany * l.rows_many : 0);
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

    void reserve(const PlanLimits &l)
    {
        few.reserve(l.cap_few);
        many.reserve(l.cap_many);
        whole.reserve(std::max(l.cap_few, l.cap_many));
        groups.reserve(l.cap_groups);
        append.reserve(l.cap_append);
    }
};

// Splits the pieces in `whole` (tile0 = 0, tile1 = all tiles) over the keys.  Fewer pieces than
// workgroups that run at once: the smallest share of tiles whose cuts do not outnumber them, so
// that all run in one go; otherwise only pieces longer than the even share are cut.  Either way no more
// than 2 * slots parts are cut: a piece of t tiles gives at most t / share + 1 <= 2 t / share, and the
// sum of t / share is at most slots.  A part shorter than min_tiles is not worth its partial
// result's trip.
inline void split_class(Plan &p, std::vector<AttnItem> &out, const PlanLimits &l, int32_t rows_of_piece,
                        int64_t slots, int64_t min_tiles, int64_t *prow)
{
    int64_t total = 0, longest = 0;
    for (const AttnItem &it : p.whole) total += it.tile1, longest = std::max<int64_t>(longest, it.tile1);
    int64_t share = std::max(min_tiles, (total + slots - 1) / slots);
    if ((int64_t)p.whole.size() < slots) {
        int64_t hi = std::max(share, longest);  // no cut at all: fits
        while (share < hi) {
            const int64_t mid = (share + hi) / 2;
            int64_t n = 0;
            for (const AttnItem &it : p.whole) n += std::max<int64_t>(1, (it.tile1 + mid - 1) / mid);
            if (n <= slots) hi = mid;
            else share = mid + 1;
        }
    }
    for (const AttnItem &it : p.whole) {
        const int64_t n = (it.tile1 + share - 1) / share;
        if (n <= 1) {
            out.push_back(it);
            continue;
        }
        const int32_t rows = (int32_t)std::min<int64_t>(rows_of_piece, (int64_t)it.q_len * l.group - it.row0);
        for (int32_t r = 0; r < rows; r += KVX_JOIN_ROWS)
            p.groups.push_back(AttnGroup{(int32_t)*prow + r, (int32_t)n, rows_of_piece,
                                         std::min(KVX_JOIN_ROWS, rows - r), it.q_begin, it.q_len, it.head,
                                         it.row0 + r});
        for (int64_t k = 0; k < n; ++k) {
            AttnItem part = it;
            part.tile0 = (int32_t)(it.tile1 * k / n);
            part.tile1 = (int32_t)(it.tile1 * (k + 1) / n);
            part.prow = (int32_t)*prow;
            *prow += rows_of_piece;
            out.push_back(part);
        }
    }
    // longest first, so that the last workgroups to start are the short ones
    std::stable_sort(out.begin(), out.end(), [](const AttnItem &a, const AttnItem &b) {
        return a.tile1 - a.tile0 > b.tile1 - b.tile0;
    });
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
    for (int cls = 0; cls < 2; ++cls) {
        const bool few = cls == 0;
        const int32_t step = few ? KVX_ROWS_FEW : l.rows_many;
        p.whole.clear();
        for (int32_t i = 0; i < n; ++i) {
            const kv_seq &s = seqs[i];
            const int64_t rows = (int64_t)s.q_len * l.group;
            if (rows == 0 || (rows <= KVX_ROWS_FEW) != few) continue;
            for (int64_t r = 0; r < rows; r += step) {
                const int32_t t0 = (int32_t)(r / l.group);
                const int32_t t1 = (int32_t)((std::min(rows, r + step) - 1) / l.group);
                const int32_t first = (int32_t)(s.kv_len - s.q_len);
                const KeyWalk w =
                    key_walk((int32_t)s.kv_len, s.prefix_len, l.window, l.full, first + t0, first + t1);
                AttnItem it{};
                it.table = s.block_table;
                it.kv_len = (int32_t)s.kv_len;
                it.q_begin = (int32_t)s.q_begin;
                it.q_len = s.q_len;
                it.prefix = s.prefix_len;
                it.row0 = (int32_t)r;
                it.tile1 = w.n_tiles;
                it.prow = -1;
                for (it.head = 0; it.head < l.heads; ++it.head) p.whole.push_back(it);
            }
        }
        split_class(p, few ? p.few : p.many, l, step, few ? l.slots_few : kSlotsMany, few ? 2 : 4, &prow);
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
