// Runs the kernels' rule of counting and joining shared items
// (csrc/join_rule.h) over every order in which CTAs can begin, count their
// parts and look at the counts, and checks that every share of every item is
// joined exactly once, and that no CTA waits for one that has not begun.
// Prints "ok <layouts> <states>", or the first layout that fails.
#include <stdio.h>

#include <set>
#include <vector>

#include "join_rule.h"

using namespace w4a16;

struct Item {
    int first, parts, tiles;  // shared by CTAs first .. first + parts - 1, counted in by `tiles` threads of each
};
struct Layout {
    int ctas, joiners;  // at most so many of an item's CTAs have a share
    std::vector<Item> items;
};

// A CTA: begins; each of its two counting threads counts its items in, in
// order; then, item by item, it looks (waits, if it may) and joins.
struct Cta {
    bool begun = false;
    int counted[2] = {0, 0}, looked = 0;
    bool waits[2] = {true, true};
    unsigned seen[2][2] = {{0, 0}, {0, 0}};  // [its item][thread]
};
struct State {
    int begun = 0;
    std::vector<Cta> ctas;
    std::vector<unsigned> arrived;
    std::vector<std::vector<int>> joined;  // [item][share]: how often
    std::vector<int> key() const {
        std::vector<int> k{begun};
        for (const Cta &c : ctas)
            for (int v : {(int)c.begun, c.counted[0], c.counted[1], c.looked, (int)c.waits[0], (int)c.waits[1],
                          (int)c.seen[0][0], (int)c.seen[0][1], (int)c.seen[1][0], (int)c.seen[1][1]})
                k.push_back(v);
        for (unsigned a : arrived) k.push_back((int)a);
        for (const auto &j : joined) k.insert(k.end(), j.begin(), j.end());
        return k;
    }
};

static long long g_states = 0;
static const char *g_why = nullptr;

struct Run {
    const Layout &l;
    std::vector<std::vector<int>> mine;  // items of each CTA
    std::set<std::vector<int>> been;

    explicit Run(const Layout &layout) : l(layout), mine(layout.ctas) {
        for (int i = 0; i < (int)l.items.size(); ++i)
            for (int c = l.items[i].first; c < l.items[i].first + l.items[i].parts; ++c) mine[c].push_back(i);
    }
    int shares(int item) const { return l.items[item].parts < l.joiners ? l.items[item].parts : l.joiners; }

    bool go(const State &s) {
        if (!been.insert(s.key()).second) return true;
        ++g_states;
        bool moved = false, left = false;
        for (int c = 0; c < l.ctas; ++c) {
            const Cta &cta = s.ctas[c];
            if (!cta.begun) {
                State n = s;
                n.ctas[c].begun = true;
                ++n.begun;
                moved = left = true;
                if (!go(n)) return false;
                continue;
            }
            bool counting = false;
            for (int t = 0; t < 2; ++t) {
                int k = cta.counted[t];
                while (k < (int)mine[c].size() && t >= l.items[mine[c][k]].tiles) ++k;
                if (k >= (int)mine[c].size()) continue;
                counting = moved = left = true;
                const int item = mine[c][k];
                State n = s;
                const unsigned mark = part_mark(s.begun == l.ctas, n.ctas[c].waits[t]);
                n.arrived[item] += mark;
                n.ctas[c].seen[k][t] = n.arrived[item];
                n.ctas[c].counted[t] = k + 1;
                if (!go(n)) return false;
            }
            if (counting || cta.looked == (int)mine[c].size()) continue;
            left = true;
            const int item = mine[c][cta.looked], index = c - l.items[item].first;
            const unsigned all = l.items[item].parts * l.items[item].tiles, *seen = cta.seen[cta.looked];
            const unsigned own = (seen[1] & kCountMask) > (seen[0] & kCountMask) ? seen[1] : seen[0];
            const bool waits = index < shares(item) && cta.waits[0];
            if (waits && s.begun != l.ctas) {
                g_why = "a CTA waits while another has not begun";
                return false;
            }
            if (waits && (s.arrived[item] & kCountMask) < all) continue;  // not yet
            moved = true;
            bool failed;
            const int mode = join_mode(waits ? s.arrived[item] : own, own, waits, all, failed);
            if (failed) {
                g_why = "a count taken for a failure";
                return false;
            }
            State n = s;
            for (int x = 0; x < shares(item); ++x)
                if (mode == kJoinAll || (mode == kJoinShare && x == index)) ++n.joined[item][x];
            ++n.ctas[c].looked;
            if (!go(n)) return false;
        }
        if (!moved && left) {
            g_why = "CTAs wait for one another";
            return false;
        }
        if (!left)
            for (const auto &j : s.joined)
                for (int times : j)
                    if (times != 1) {
                        g_why = times ? "a share joined twice" : "a share never joined";
                        return false;
                    }
        return true;
    }
    bool all() {
        State s;
        s.ctas.resize(l.ctas);
        s.arrived.assign(l.items.size(), 0);
        for (int i = 0; i < (int)l.items.size(); ++i) s.joined.push_back(std::vector<int>(shares(i), 0));
        return go(s);
    }
};

static bool waits_end() {
    // A count that stays below the parts: given up once the limit is over, with a failure and nothing joined.
    for (unsigned have : {0u, 1u, 5u, kWontWait + 5u}) {
        unsigned long long ns = 1000, looks = 0;
        const unsigned now = await_count(6, 2000, [&] { ++looks; return have; }, [&] { return ns += 500; });
        bool failed = false;
        if (now != have || ns - 1500 <= 2000 || ns - 1500 > 2500 || looks != 64 * (ns - 1000) / 500 ||
            join_mode(now, have, true, 6, failed) != kJoinNothing || !failed)
            return false;
    }
    // Reached at some look: no failure.
    unsigned looks = 0;
    bool failed = true;
    const unsigned now = await_count(6, 2000, [&] { return ++looks > 100 ? 6u : 5u; }, [] { return 7ull; });
    if (now != 6 || looks != 101 || join_mode(now, 3, true, 6, failed) != kJoinShare || failed) return false;
    // More counts, or more marks, than parts: a workspace that was not zeroed.
    return join_mode(7, 7, true, 6, failed) == kJoinNothing && failed &&
           join_mode(7 * kWontWait + 6, 6, false, 6, failed) == kJoinNothing && failed;
}

int main() {
    if (!waits_end()) {
        printf("a wait does not end as it should\n");
        return 1;
    }
    std::vector<std::vector<Item>> chains = {
        {{0, 2, 1}, {1, 2, 1}}, {{0, 3, 1}}, {{0, 2, 1}, {1, 3, 1}}, {{0, 3, 1}, {2, 2, 1}}, {{0, 2, 1}, {1, 2, 1}, {2, 2, 1}},
        {{0, 2, 2}, {1, 2, 2}}, {{0, 2, 2}, {1, 2, 1}}, {{0, 2, 1}, {1, 2, 2}}, {{0, 3, 2}}};
    int layouts = 0;
    for (const auto &items : chains)
        for (int more = 0; more < 2; ++more)  // a CTA that shares nothing, and may begin late
            for (int joiners = 1; joiners <= 3; ++joiners) {
                Layout l{items.back().first + items.back().parts + more, joiners, items};
                Run run(l);
                if (!run.all()) {
                    printf("%s: %d CTAs, %d joiners, items", g_why, l.ctas, joiners);
                    for (const Item &i : items) printf(" (first %d, parts %d, tiles %d)", i.first, i.parts, i.tiles);
                    printf("\n");
                    return 1;
                }
                ++layouts;
            }
    printf("ok %d %lld\n", layouts, g_states);
    return 0;
}
