// Every interleaving of a team's warps over a few rows, with csrc/give_up.h as the
// kernels use it: wait for the row (it lands, or runs out and is marked), arrive at the
// team's barrier, read the mark behind it, leave or go on. With `next`, a warp that
// goes on may also mark the row after (as the cluster's warps do), and a warp that has
// given up walks on to the last row without waiting. Exit status 0: no interleaving
// stops before every warp has ended, and all warps give up at the same row.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "give_up.h"

namespace {

int warps, rows;
bool next;

enum Where : int { kWaits, kAtBarrier, kBehind, kEnded };

struct State {
    unsigned int late[2];
    std::vector<int> where, row, gave_up_at;  // -1: has not
    std::vector<int> key() const {
        std::vector<int> k{static_cast<int>(late[0]), static_cast<int>(late[1])};
        for (int w = 0; w < warps; ++w) k.insert(k.end(), {where[w], row[w], gave_up_at[w]});
        return k;
    }
};

std::set<std::vector<int>> seen;
bool hung = false, differ = false;

void walk(const State& s);

template <typename F>
void step(const State& s, F change) {
    State n = s;
    rmsn::GiveUp g;
    g.late[0] = n.late[0];
    g.late[1] = n.late[1];
    change(n, g);
    n.late[0] = g.late[0];
    n.late[1] = g.late[1];
    walk(n);
}

void walk(const State& s) {
    if (!seen.insert(s.key()).second) return;
    bool moved = false, ended = true;
    int arrived = 0;
    for (int w = 0; w < warps; ++w) {
        ended &= s.where[w] == kEnded;
        arrived += s.where[w] == kAtBarrier;
    }
    if (arrived == warps) {  // the barrier opens for all of them
        moved = true;
        step(s, [&](State& n, rmsn::GiveUp&) {
            for (int w = 0; w < warps; ++w) n.where[w] = kBehind;
        });
    }
    for (int w = 0; w < warps; ++w) {
        if (s.where[w] == kWaits) {
            moved = true;
            for (int out = 0; out < 2; ++out) {
                if (out && s.gave_up_at[w] >= 0) continue;  // does not wait any more
                step(s, [&](State& n, rmsn::GiveUp& g) {
                    if (out) g.mark(n.row[w]);
                    n.where[w] = kAtBarrier;
                });
            }
        } else if (s.where[w] == kBehind) {
            moved = true;
            for (int mark_next = 0; mark_next <= (next ? 1 : 0); ++mark_next)
                step(s, [&](State& n, rmsn::GiveUp& g) {
                    if (n.gave_up_at[w] < 0 && g.at(n.row[w])) n.gave_up_at[w] = n.row[w];
                    if (mark_next) g.mark(n.row[w] + 1);
                    const bool leave = n.gave_up_at[w] >= 0 && !next;
                    n.where[w] = leave || ++n.row[w] == rows ? kEnded : kWaits;
                });
        }
    }
    if (!moved && !ended) hung = true;
    if (ended)
        for (int w = 1; w < warps; ++w) differ |= s.gave_up_at[w] != s.gave_up_at[0];
}

}  // namespace

int main(int argc, char** argv) {
    if (argc != 4) return 2;
    warps = std::atoi(argv[1]);
    rows = std::atoi(argv[2]);
    next = std::atoi(argv[3]) != 0;
    State s;
    rmsn::GiveUp g;
    g.clear();
    s.late[0] = g.late[0];
    s.late[1] = g.late[1];
    s.where.assign(warps, kWaits);
    s.row.assign(warps, 0);
    s.gave_up_at.assign(warps, -1);
    walk(s);
    std::printf("%d warps, %d rows: %zu states%s%s\n", warps, rows, seen.size(), hung ? ", one of them hangs" : "",
                differ ? ", warps give up at different rows" : "");
    return hung || differ ? 1 : 0;
}
