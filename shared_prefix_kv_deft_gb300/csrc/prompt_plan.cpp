// prompt_plan.cpp -- host planner of the prompt step: query tiles, splits of
// long key ranges, and the units each CTA runs.
//
// A prompt is the last m tokens of a node; its rows (m tokens x GQA group,
// token-major, so that the heads of a group share every K and V tile) are
// cut into tiles of floor(128 / group) tokens, and neighbouring tiles are
// paired (tensor-core work of one hides under the softmax of the other).  A
// tile reads the pages of the path in one order: the ancestors' from the
// node's parent up to its root, then the node's own up to its last row's
// token (causal), so the masked pages come last.
//
// Units (item x KV head) are dealt to kPromptCtas CTAs by list scheduling
// on an estimated cost: in order, each to the CTA that is free first.  A
// dealt list needs no work queue, so steps of one plan may run at the same
// time.  With few units a CTA the order is costliest item first over all
// heads, which balances best; with many it is head by head (each costliest
// item first): the CTAs running at a time then read few heads' K and V,
// which stay in L2, and the last head's smallest items fill the gaps.
//
// When a few units would leave SMs idle or one unit would outlast the rest,
// the page ranges of the items are cut into pieces whose partial results a
// second launch merges by log-sum-exp.  The cut is chosen by simulating the
// deal for a few piece sizes and taking the shortest, the pieces' fp32 rows
// and the merge counted.  Units of a few near lengths that do not divide among
// the CTAs (the next chunks of several requests) are levelled by cutting only
// the shortest items, a twentieth of the work, finely.  A length bound picks
// them, so a batch of one single length is not levelled (eight chunks of 512
// at 8192 tokens, 32/8 heads: the longest CTA has 1.18 times the mean; 160
// equal units: 1.9 times).  Cutting a 4096-token
// prompt of 16 heads into 640 units instead of 256 moved 75 MB of partials
// and cost more than it gained (95 us against 55 us).
#include <algorithm>
#include <vector>

#include "prompt_internal.h"

namespace deft {
namespace {

// Estimated costs in KV tiles of a pair of query tiles (1.33 us each).
constexpr double kCostSingle = 0.75;  // a KV tile against one query tile
constexpr double kCostUnit = 2.0;     // a unit's start and end
constexpr double kCostPiece = 1.5;    // a piece's fp32 rows (twice a bf16 tile's bytes, row by row)
constexpr double kCostMerge = 3.0;    // the merge launch
constexpr double kCostSlot = 1e-4;    // a partial row, written and read once through L2
constexpr int32_t kMinPieceTiles = 4; // shortest piece
// Above, no split is looked for: so many units of like length balance by
// themselves, and each simulation costs host time in their number.  One far
// longer unit among them is not cut and outlasts the rest (160 single tokens
// of 8 heads, one at 131072 tokens and the others at 2048: 4.9 times the mean
// load; a 512-token chunk at 65536 beside 200 such tokens: 1.4 times).
constexpr int64_t kMaxSimUnits = 8 * kPromptCtas;
constexpr int64_t kMaxCostOrder = 16 * kPromptCtas; // above, units go head by head (few-shot prefill, 10 units a CTA: 442 us by cost, 449 by head)

int32_t pages_of(int64_t tokens) { return (int32_t)((tokens + kPageSize - 1) / kPageSize); }
int32_t tiles_of(int32_t pages) { return (pages + kPromptTilePages - 1) / kPromptTilePages; }

// An item before its page range is cut.
struct Proto {
    PromptItem it;
    int32_t pages_a, pages_b;   // pages tile A / B reads from the path's first page on
    int32_t prompt_above;       // pages of the ancestors
    int32_t tiles() const { return tiles_of(std::max(pages_a, pages_b)); }
    double tile_cost() const { return it.tok_b > 0 ? 1.0 : kCostSingle; }
};

// Where ranges are cut: above `cap` tiles, and above `fine` where there are at
// most `below`.
struct Cuts {
    int32_t cap = INT32_MAX, below = 0, fine = INT32_MAX;
};
int32_t pieces_of(const Proto &p, const Cuts &c)
{
    return 1 + (p.tiles() - 1) / (p.tiles() <= c.below ? std::min(c.cap, c.fine) : c.cap);
}

// The CTAs by the time they are free, earliest first (equal times: lowest
// number): a tree of minima over one key a CTA, its time in 1/4096 tiles
// above its number, so that giving the first more work is eight minima.
struct Deal {
    static constexpr int32_t kLeaves = 256;
    static_assert(kPromptCtas <= kLeaves, "a CTA's number in eight bits");
    uint64_t key[2 * kLeaves];
    uint64_t end = 0;
    Deal()
    {
        for (int32_t c = 0; c < kLeaves; ++c)
            key[kLeaves + c] = c < kPromptCtas ? (uint64_t)c : UINT64_MAX;
        for (int32_t i = kLeaves - 1; i > 0; --i)
            key[i] = std::min(key[2 * i], key[2 * i + 1]);
    }
    // The CTA that takes a unit of this cost.
    int32_t take(uint64_t cost)
    {
        const int32_t id = (int32_t)(key[1] & 255);
        uint64_t x = key[1] + (cost << 8);
        end = std::max(end, x >> 8);
        int32_t i = kLeaves + id;
        key[i] = x;
        for (; i > 1; i >>= 1) {
            x = std::min(x, key[i ^ 1]);
            key[i >> 1] = x;
        }
        return id;
    }
    static uint64_t units(double tiles) { return (uint64_t)(tiles * 4096.0); }
};

bool head_major(size_t items, int32_t heads) { return (int64_t)items * heads > kMaxCostOrder; }

// Length of the deal (costliest item first) when ranges are cut so.
double simulate(const std::vector<Proto> &protos, int32_t heads, int32_t group, const Cuts &cuts)
{
    std::vector<double> cost;
    double slots = 0;
    for (const Proto &p : protos) {
        const int32_t n = pieces_of(p, cuts), t = (p.tiles() + n - 1) / n;
        if (n > 1)
            slots += (double)n * (p.it.tok_a + p.it.tok_b) * group * heads;
        for (int32_t i = 0; i < n; ++i)
            cost.push_back(kCostUnit + (n > 1 ? kCostPiece : 0.0) + t * p.tile_cost());
    }
    std::sort(cost.begin(), cost.end(), std::greater<double>());
    Deal deal;
    for (const double c : cost) {
        const uint64_t x = Deal::units(c);
        for (int32_t h = 0; h < heads; ++h)
            deal.take(x);
    }
    return (double)deal.end / 4096.0 + (slots > 0 ? kCostMerge + kCostSlot * slots : 0.0);
}

}  // namespace

int build_prompt_plan(const int32_t *parent, const int32_t *node_len, int32_t num_nodes, const int32_t *prompt_node,
                      const int32_t *prompt_len, int32_t num_prompts, int32_t num_kv_heads, int32_t gqa_group,
                      deft_prompt_plan_t *p)
{
    if (!node_len || num_nodes < 1 || num_prompts < 0 || (num_prompts > 0 && !prompt_node) || num_kv_heads < 1 ||
        num_kv_heads > 65535 || gqa_group < 1 || gqa_group > kMmaMaxRows)
        return DEFT_EINVAL;
    for (int32_t n = 0; n < num_nodes; ++n) {
        if (node_len[n] < 0)
            return DEFT_EINVAL;
        if (parent && (parent[n] < -1 || parent[n] >= num_nodes))
            return DEFT_ERANGE;
    }
    // Nearest ancestor with tokens and the pages and tokens above each node,
    // parents first; a node met again on the way up belongs to a cycle.
    p->nodes.assign(2 * (size_t)num_nodes, -1);
    std::vector<int64_t> above(num_nodes, -1), tok_above(num_nodes, -1);
    std::vector<int32_t> way;
    std::vector<uint8_t> seen(num_nodes, 0);   // 1: on the way, 2: done
    for (int32_t n = 0; n < num_nodes; ++n) {
        way.clear();
        int32_t a = n;
        while (a >= 0 && seen[a] == 0) {
            seen[a] = 1;
            way.push_back(a);
            a = parent ? parent[a] : -1;
        }
        if (a >= 0 && seen[a] == 1)
            return DEFT_ECYCLE;
        for (auto it = way.rbegin(); it != way.rend(); ++it) {
            const int32_t x = *it, up = parent ? parent[x] : -1;
            const int32_t from = up < 0 ? -1 : node_len[up] > 0 ? up : p->nodes[2 * (size_t)up];
            p->nodes[2 * (size_t)x] = from;
            p->nodes[2 * (size_t)x + 1] = node_len[x];
            above[x] = from < 0 ? 0 : above[from] + pages_of(node_len[from]);
            tok_above[x] = from < 0 ? 0 : tok_above[from] + node_len[from];
            if (above[x] + pages_of(node_len[x]) > (1 << 25) - 1)
                return DEFT_EUNSUPPORTED;
            seen[x] = 2;
        }
    }
    p->num_nodes = num_nodes;
    p->num_prompts = num_prompts;
    p->num_kv_heads = num_kv_heads;
    p->gqa_group = gqa_group;
    p->items.clear();
    p->cta_unit.clear();
    p->merges.clear();
    p->part_slots = 0;
    deft_prompt_stats st{};

    const int32_t tile_tok = kPromptRows / gqa_group;
    std::vector<Proto> protos;
    int64_t rows = 0, pair_tokens = 0;
    for (int32_t i = 0; i < num_prompts; ++i) {
        const int32_t n = prompt_node[i];
        if (n < 0 || n >= num_nodes)
            return DEFT_ERANGE;
        const int32_t L = node_len[n];
        const int32_t m = !prompt_len || prompt_len[i] == -1 ? L : prompt_len[i];
        if (m < 0 || m > L)
            return DEFT_ERANGE;
        // Refused here, before the records of such a batch are made.
        const int64_t pairs = ((int64_t)m + 2 * tile_tok - 1) / (2 * tile_tok);
        if (((int64_t)protos.size() + pairs) * num_kv_heads > INT32_MAX / 8 || rows + m > INT32_MAX)
            return DEFT_EUNSUPPORTED;
        for (int32_t t = 0; t < m; t += 2 * tile_tok) {
            Proto q{};
            q.it.row0 = (int32_t)(rows + t);
            q.it.tok_a = std::min(tile_tok, m - t);
            q.it.tok_b = std::min(tile_tok, m - t - q.it.tok_a);
            q.it.pos0 = L - m + t;
            q.it.node = n;
            q.it.part0 = -1;
            q.prompt_above = (int32_t)above[n];
            q.pages_a = (int32_t)above[n] + pages_of((int64_t)q.it.pos0 + q.it.tok_a);
            q.pages_b = q.it.tok_b ? (int32_t)above[n] + pages_of((int64_t)q.it.pos0 + q.it.tok_a + q.it.tok_b) : 0;
            protos.push_back(q);
        }
        rows += m;
        // Tokens seen: those above (exactly, not in pages), then 1 .. m of
        // the node's last m and all before them.
        pair_tokens += (int64_t)m * (tok_above[n] + L - m) + (int64_t)m * (m + 1) / 2;
    }
    p->num_rows = (int32_t)rows;

    // Where to cut, if a cut can gain more than its merge costs.
    Cuts cuts;
    const int64_t whole = (int64_t)protos.size() * num_kv_heads;
    if (whole <= kMaxSimUnits && !protos.empty()) {
        double total = 0;
        int32_t longest = 0;
        for (const Proto &q : protos) {
            total += q.tiles() * q.tile_cost();
            longest = std::max(longest, q.tiles());
        }
        const double even = total * num_kv_heads / kPromptCtas;
        double best = simulate(protos, num_kv_heads, gqa_group, cuts);
        const double least = even + kCostUnit * (double)whole / kPromptCtas + kCostMerge;
        auto try_cuts = [&](const Cuts &c) {
            const double t = simulate(protos, num_kv_heads, gqa_group, c);
            if (t < best) {
                best = t;
                cuts = c;
            }
        };
        for (const double part : {1.4, 1.2, 1.0, 0.6}) {
            Cuts c;
            c.cap = std::max(kMinPieceTiles, (int32_t)(even * part + 0.999));
            if (best > least && c.cap < longest)
                try_cuts(c);
        }
        if (best > least && cuts.cap == INT32_MAX) {
            // The shortest items, a twentieth of the work, in small pieces.
            std::vector<int32_t> tiles;
            for (const Proto &q : protos)
                tiles.push_back(q.tiles());
            std::sort(tiles.begin(), tiles.end());
            Cuts c;
            double below = 0;
            for (size_t i = 0; i < tiles.size() && below < 0.05 * total; ++i) {
                c.below = tiles[i];
                below += tiles[i];
            }
            c.fine = std::max(kMinPieceTiles, (int32_t)(even * 0.07 + 0.999));
            if (c.fine < c.below)
                try_cuts(c);
        }
    }

    // The items: pieces of equal length, whole KV tiles.
    std::vector<std::pair<double, PromptItem>> cut;
    for (Proto &q : protos) {
        const int32_t n = pieces_of(q, cuts), t = (q.tiles() + n - 1) / n;
        const int32_t all = std::max(q.pages_a, q.pages_b);
        const int32_t item_rows = (q.it.tok_a + q.it.tok_b) * gqa_group;
        const int64_t piece_slots = (int64_t)item_rows * num_kv_heads;
        int32_t made = 0;
        const int64_t part0 = p->part_slots;
        // The page the next piece starts at, walked along the path.
        int32_t node = q.prompt_above > 0 ? p->nodes[2 * (size_t)q.it.node] : q.it.node, first = 0;
        for (int32_t begin = 0; begin < all; begin += t * kPromptTilePages) {
            const int32_t end = std::min(all, begin + t * kPromptTilePages);
            PromptItem it = q.it;
            it.pages = end - begin;
            it.tiles_a = tiles_of(std::max(0, std::min(end, q.pages_a) - begin));
            it.tiles_b = tiles_of(std::max(0, std::min(end, q.pages_b) - begin));
            it.start_node = node;
            it.start_page = first;
            if (n > 1) {
                if (part0 + (made + 1) * piece_slots > INT32_MAX)
                    return DEFT_EUNSUPPORTED;
                it.part0 = (int32_t)(part0 + made * piece_slots);
            }
            ++made;
            cut.emplace_back(kCostUnit + (n > 1 ? kCostPiece : 0.0) + std::max(it.tiles_a, it.tiles_b) * q.tile_cost(), it);
            for (int32_t left = end - begin; left > 0 && end < all;) {
                const int32_t here = node == q.it.node ? INT32_MAX : pages_of(node_len[node]) - first;
                const int32_t step = std::min(left, here);
                first += step;
                left -= step;
                if (step == here) {
                    node = p->nodes[2 * (size_t)node];
                    if (node < 0)
                        node = q.it.node;
                    first = 0;
                }
            }
        }
        if (n > 1) {
            p->part_slots = part0 + made * piece_slots;
            p->merges.push_back(PromptMerge{q.it.row0, q.it.tok_a + q.it.tok_b, (int32_t)part0, made});
        }
    }
    std::stable_sort(cut.begin(), cut.end(), [](const auto &a, const auto &b) { return a.first > b.first; });
    if ((int64_t)cut.size() * num_kv_heads > INT32_MAX)
        return DEFT_EUNSUPPORTED;

    // The deal.
    const size_t units = cut.size() * num_kv_heads;
    const bool by_head = head_major(cut.size(), num_kv_heads);
    auto each_unit = [&](auto &&f) {   // in the order of the deal
        const size_t items = cut.size(), heads = (size_t)num_kv_heads;
        for (size_t x = 0; x < (by_head ? heads : items); ++x)
            for (size_t y = 0; y < (by_head ? items : heads); ++y)
                f(by_head ? y : x, by_head ? x : y);
    };
    std::vector<uint8_t> owner(units);
    p->cta_off.assign(kPromptCtas + 1, 0);
    Deal deal;
    size_t u = 0;
    each_unit([&](size_t i, size_t) {
        const int32_t c = deal.take(Deal::units(cut[i].first));
        owner[u++] = (uint8_t)c;
        ++p->cta_off[c + 1];
    });
    for (int32_t c = 0; c < kPromptCtas; ++c)
        p->cta_off[c + 1] += p->cta_off[c];
    std::vector<int32_t> at(p->cta_off.begin(), p->cta_off.end() - 1);
    p->cta_unit.resize(units);
    u = 0;
    each_unit([&](size_t i, size_t h) {
        p->cta_unit[at[owner[u++]]++] = (int32_t)(i * num_kv_heads + h);
    });
    p->items.reserve(cut.size());
    for (const auto &c : cut)
        p->items.push_back(c.second);

    st.num_nodes = num_nodes;
    st.num_prompts = num_prompts;
    st.num_rows = (int32_t)rows;
    st.num_items = (int32_t)p->items.size();
    st.num_units = (int32_t)p->cta_unit.size();
    st.num_split_items = (int32_t)p->merges.size();
    st.ctas = (int32_t)std::min<size_t>(kPromptCtas, p->cta_unit.size());
    st.pair_tokens = pair_tokens;
    st.partial_slots = p->part_slots;
    p->stats = st;
    return DEFT_OK;
}

}  // namespace deft
