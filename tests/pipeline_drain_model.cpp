// A model of the products' ring of stages, run with random interleavings and
// waits that give up at random, to check that the drain ends with no load in
// flight.
//
//   pipeline_drain_model <ctas> <storing roles per CTA> <stages> <runs> <drain>
//
// drain 1: the counts' rule of pipeline_drain.h.  drain 0: only where the
// leader's load role itself gave up, which is the mistake that the rule
// replaces.  Prints the runs that gave up and those that left loads in flight.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pipeline_drain.h"

using namespace bsq;

struct Barrier {
    int count, pending, phase = 0;
    long tx = 0;
    explicit Barrier(int n) : count(n), pending(n) {}
    void settle() {
        if (pending == 0 && tx == 0) {
            ++phase;
            pending = count;
        }
    }
    void arrive(long expect = 0) {
        if (pending <= 0) {
            std::printf("an arrival too many\n");
            std::exit(2);
        }
        tx += expect;
        --pending;
        settle();
    }
    void land(long bytes) {
        tx -= bytes;
        settle();
    }
};

struct Load {
    int cta, j;
    long bytes;
};

static std::mt19937_64 rng(1);
static int pick(int n) { return (int)(rng() % (uint64_t)n); }

struct Run {
    int ctas, roles, stages, steps, limit;  // limit: 1 in this many failed waits gives up
    std::vector<Barrier> full;
    std::vector<std::vector<int>> freed;  // [cta][stage] completed phases of the "empty" barriers
    std::vector<Load> flight;
    std::vector<int> commits;  // stages whose MMAs have been issued and not completed
    std::vector<int> aborted;
    std::vector<long> bytes;
    std::vector<int> issued, stored, load_done, store_done;
    bool load_ok[2] = {true, true};
    int mma = 0;
    bool mma_done = false;

    Run(int c, int r, int s)
        : ctas(c), roles(r), stages(s), steps(1 + pick(4 * s)), limit(2 + pick(40)), full(s, Barrier(c * r + 1)),
          freed(c, std::vector<int>(s, 0)), aborted(c, 0), issued(c, 0), stored(c * r, 0), load_done(c, 0), store_done(c * r, 0) {
        for (int j = 0; j < steps; ++j) bytes.push_back(1 + pick(1000));
    }
    // the wait of a role of CTA c: 1 passed, 0 not yet, -1 given up
    int wait(bool passed, int c) {
        if (passed) return 1;
        if (aborted[c] || pick(limit) == 0) {
            aborted[c] = 1;
            return -1;
        }
        return 0;
    }
    bool empty_for(int c, int j) { return freed[c][j % stages] >= j / stages; }
    void load_role(int c) {
        const int j = issued[c];
        if (load_done[c]) return;
        if (j == steps) {
            load_done[c] = 1;
            return;
        }
        const int w = wait(empty_for(c, j), c);
        if (w < 0) {
            load_done[c] = 1;
            load_ok[c] = false;
        }
        if (w <= 0) return;
        Barrier& b = full[j % stages];
        if (b.phase != j / stages) {
            std::printf("a load into a stage that is not free\n");
            std::exit(2);
        }
        if (c == 0) b.arrive(ctas * bytes[j]);
        flight.push_back({c, j, bytes[j]});
        ++issued[c];
    }
    void store_role(int i) {
        const int c = i / roles, j = stored[i];
        if (store_done[i]) return;
        if (j == steps) {
            store_done[i] = 1;
            return;
        }
        const int w = wait(empty_for(c, j), c);
        if (w < 0) store_done[i] = 1;
        if (w <= 0) return;
        full[j % stages].arrive();
        ++stored[i];
    }
    void mma_role() {
        if (mma_done) return;
        if (mma == steps) {
            mma_done = true;
            return;
        }
        const int w = wait(full[mma % stages].phase > mma / stages, 0);
        if (w < 0) mma_done = true;
        if (w <= 0) return;
        commits.push_back(mma % stages);
        ++mma;
    }
    void hardware() {
        if (!flight.empty() && pick(3) == 0) {
            const int i = pick((int)flight.size());
            const Load l = flight[i];
            flight.erase(flight.begin() + i);
            full[l.j % stages].land(l.bytes);
        }
        if (!commits.empty() && pick(3) == 0) {
            for (auto& f : freed) ++f[commits.front()];
            commits.erase(commits.begin());
        }
    }
    bool stopped() {
        bool s = mma_done;
        for (int d : load_done) s = s && d;
        for (int d : store_done) s = s && d;
        return s;
    }
};

int main(int argc, char** argv) {
    if (argc != 6) return 2;
    const int ctas = std::atoi(argv[1]), roles = std::atoi(argv[2]), stages = std::atoi(argv[3]), runs = std::atoi(argv[4]);
    const bool rule = std::atoi(argv[5]) != 0;
    long gave_up = 0, left = 0;
    for (int n = 0; n < runs; ++n) {
        Run r(ctas, roles, stages);
        const int actors = ctas + ctas * roles + 2;
        while (!r.stopped()) {
            const int a = pick(actors);
            if (a < ctas) r.load_role(a);
            else if (a < ctas + ctas * roles) r.store_role(a - ctas);
            else if (a == actors - 2) r.mma_role();
            else r.hardware();
        }
        bool any = false;
        for (int a : r.aborted) any = any || a;
        gave_up += any;
        if (!any) {
            left += !r.flight.empty();
            continue;
        }
        if (!rule) {
            // its waits end after the bytes have landed, or at a limit long after
            if (r.load_ok[0]) left += !r.flight.empty();
            else for (const Load& l : r.flight) {
                if (l.j >= r.issued[0] || l.j < r.issued[0] - stages) {  // not waited for
                    ++left;
                    break;
                }
            }
            continue;
        }
        const int first = drain_first(r.issued.data(), ctas, stages), last = drain_last(r.issued.data(), ctas);
        for (const Load& l : r.flight)
            if (l.j < first || l.j >= last) {
                std::printf("a load outside the k-steps waited for\n");
                return 2;
            }
        for (int j = first; j < last; ++j) {
            const PhaseDebt d = phase_debt(j, r.issued.data(), ctas, (uint32_t)r.bytes[j], r.stored.data(), ctas * roles);
            Barrier& b = r.full[j % stages];
            if (d.expect) b.arrive(d.expect);
            if (d.complete) b.land(d.complete);
            for (uint32_t i = 0; i < d.arrivals; ++i) b.arrive();
        }
        // the leader waits for the phases, with the hardware at work
        for (int j = first; j < last; ++j)
            for (long tries = 0; r.full[j % stages].phase <= j / stages; ++tries) {
                if (r.flight.empty() || tries > 1000000) {
                    std::printf("k-step %d of [%d, %d) never completes\n", j, first, last);
                    return 2;
                }
                const int i = pick((int)r.flight.size());
                const Load l = r.flight[i];
                r.flight.erase(r.flight.begin() + i);
                r.full[l.j % stages].land(l.bytes);
            }
        left += !r.flight.empty();
    }
    std::printf("gave up %ld left in flight %ld\n", gave_up, left);
    return 0;
}
