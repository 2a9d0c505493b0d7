// A simulation of the shared-prefix kernel's loaders, product warps and softmax warps
// over its barriers: which slot each takes and waits for (pda_ring.h), with copies that
// land, and products that complete, at random times.  It fails where a slot is taken
// before it is filled, filled before it is free, or where nobody can go on.
//
// usage: prefix_ring_sim RUNS SEED RING
//   RING  own: as the kernel is; one: the streams' alternate tiles in one ring of slots;
//         eager: loaders that do not wait for a segment's products before the next one
//         (two rings that are known to be wrong, to see that the simulation can tell)
// Prints the first failure, exit status 1; or the number of runs, 0.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <coroutine>
#include <deque>
#include <memory>
#include <random>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "pda_ring.h"

namespace {

struct Process {
    struct promise_type {
        std::exception_ptr error;
        Process get_return_object() { return Process{std::coroutine_handle<promise_type>::from_promise(*this)}; }
        std::suspend_always initial_suspend() noexcept { return {}; }
        std::suspend_always final_suspend() noexcept { return {}; }
        void return_void() {}
        void unhandled_exception() { error = std::current_exception(); }
    };
    std::coroutine_handle<promise_type> h;
    explicit Process(std::coroutine_handle<promise_type> x) : h(x) {}
    Process(Process&& o) noexcept : h(std::exchange(o.h, {})) {}
    Process& operator=(Process&& o) noexcept { std::swap(h, o.h); return *this; }
    ~Process() { if (h) h.destroy(); }
    bool step() {  // false: done
        h.resume();
        if (h.promise().error) std::rethrow_exception(h.promise().error);
        return !h.done();
    }
};
constexpr std::suspend_always kYield{};

[[noreturn]] void wrong(const std::string& what) { throw std::runtime_error(what); }

// An mbarrier: a wait answers for a phase's parity alone.
struct Barrier {
    int count, pending;
    uint32_t phase = 0;  // completed ones
    explicit Barrier(int n) : count(n), pending(n) {}
    void arrive() {
        if (pending <= 0) wrong("too many arrivals");
        if (--pending == 0) { ++phase; pending = count; }
    }
    bool passed(uint32_t parity) const { return (phase & 1u) != parity; }
};

struct Segment { int n; bool dual; };
enum RingKind { kOwn, kOne, kEager };

// One ring for all: alternate tiles of two streams run four ahead of V, and a stream waits for its own only.
template <int SLOTS, bool TWO>
struct OneRing {
    uint32_t first = 0;
    uint32_t at(bool shared, int st, int own, bool k, int n, uint32_t& phase) const {
        const int ahead = shared ? 2 : 4, t = shared ? own : 2 * own + st;
        const int use = k ? t + std::max(0, t - ahead + 1) : t + std::min(t + ahead, n);
        phase = (first + use) / SLOTS & 1u;
        return (first + use) % SLOTS;
    }
    void next(bool, int n) { first += 2 * n; }
};
template <int SLOTS, bool TWO>
struct OwnRing {
    pda::PrefixRing<SLOTS, TWO> ring;
    uint32_t at(bool shared, int st, int own, bool k, int n, uint32_t& phase) const {
        const int items = shared ? n : (n - st + 1) / 2;
        return ring.slot(shared, st, k ? ring.k_use(own) : ring.v_use(own, items), phase);
    }
    void next(bool shared, int n) { ring.next(shared, n); }
};

// Q8: codes land, are spread by their loader, and only then is the slot full.
template <int SLOTS, bool TWO, bool Q8, class Ring>
class Run {
    static constexpr int kStreams = TWO ? 2 : 1;
    struct Slot { int seg = -1, tile = -1, halves = 0, readers = 0; bool k = false, busy = false; };

    std::mt19937 rnd;
    std::vector<Segment> segs;
    const RingKind kind;
    std::vector<Barrier> full, empty, landed, S, P, PV;
    Barrier O{kStreams}, Q{kStreams};
    Slot slots[SLOTS];
    std::vector<Process> procs;
    std::vector<int> speed;
    std::deque<std::vector<std::pair<Barrier*, int>>> products[2];  // of a stream, in order: arrivals, and a slot (or -1) they end

    int pick(std::initializer_list<int> x) { return x.begin()[rnd() % x.size()]; }

    Process copy(int at, int half, int delay, Slot want) {
        for (int i = 0; i < delay; ++i) co_await kYield;
        Slot& s = slots[at];
        if (s.seg != want.seg || s.tile != want.tile || s.k != want.k || !s.busy) wrong("a copy lands in a slot of another use");
        if (Q8) landed[2 * at + half].arrive();
        else { ++s.halves; full[at].arrive(); }
    }

    Process loader(bool k, int half) {
        Ring ring;
        uint32_t tiles = 0;
        std::deque<std::pair<int, uint32_t>> queue;  // (Q8) filled, not yet spread
        size_t si = 0;
        int t = 0;
        while (si < segs.size() || !queue.empty()) {
            bool can = si < segs.size();
            uint32_t phase = 0;
            int at = 0;
            Segment g{};
            if (can) {
                g = segs[si];
                const bool shared = g.dual || !TWO;
                const int st = shared ? 0 : t & 1, own = shared ? t : t >> 1;
                at = (int)ring.at(shared, st, own, k, g.n, phase);
                if (t == 0 && si > 0 && kind == kOwn) {
                    if (Q8 && !queue.empty()) can = O.passed((uint32_t)(si - 1) & 1u);
                    else while (!O.passed((uint32_t)(si - 1) & 1u)) co_await kYield;
                }
                if (Q8 && can && !queue.empty()) can = empty[at].passed(phase ^ 1u);
            }
            if (can) {
                while (!empty[at].passed(phase ^ 1u)) co_await kYield;
                Slot& s = slots[at];
                const bool same = s.busy && s.seg == (int)si && s.tile == t && s.k == k;  // (the other half's)
                if (s.busy && !same) wrong("a slot is filled before it is free");
                if (!same) {
                    s = Slot{};
                    s.seg = (int)si; s.tile = t; s.k = k; s.busy = true;
                }
                co_await kYield;
                procs.push_back(copy(at, half, pick({1, 3, 10, 10, 30, 30, pick({30, 30, 3000})}), s));
                speed.push_back(1);
                ++tiles;
                if (Q8) queue.push_back({at, phase});
                if (++t == g.n) {
                    ring.next(g.dual || !TWO, g.n);
                    ++si;
                    t = 0;
                }
            } else {
                const auto [c, ph] = queue.front();
                while (!landed[2 * c + half].passed(ph)) co_await kYield;
                ++slots[c].halves;
                full[c].arrive();
                queue.pop_front();
            }
            co_await kYield;
        }
    }

    void take(int at, int seg, bool k, int tile) {
        const Slot& s = slots[at];
        if (!s.busy || s.seg != seg || s.k != k || s.tile != tile) wrong("a stream takes a slot of another use");
        if (s.halves != 2) wrong("a stream takes a slot that is not full");
    }
    void release(int at, bool other) {  // a product with the slot is done; `other`: and the other stream needs none
        Slot& s = slots[at];
        s.readers += other ? kStreams : 1;
        if (s.readers == kStreams) s.busy = false;
    }

    // Products complete in order, some time after they are issued.
    Process pipe(int st) {
        while (true) {
            while (products[st].empty()) co_await kYield;
            for (int i = pick({0, 0, 1, 5, 40}); i > 0; --i) co_await kYield;
            auto done = products[st].front();
            products[st].pop_front();
            for (auto& [bar, slot] : done) {
                if (slot >= 0) release(slot, TWO && !segs[slots[slot].seg].dual);
                if (bar) bar->arrive();
                else co_return;
            }
        }
    }

    Process mma(int st) {
        Ring ring;
        uint32_t sn = 0, pn = 0;
        for (size_t si = 0; si < segs.size(); ++si) {
            const Segment g = segs[si];
            const bool shared = g.dual || !TWO, both = TWO && !g.dual;
            const int items = shared ? g.n : (g.n - st + 1) / 2;
            while (!Q.passed((uint32_t)si & 1u)) co_await kYield;
            for (int k = -2; k < items; ++k) {
                uint32_t phase;
                if (k >= 0) {
                    const int at = (int)ring.at(shared, st, k, false, g.n, phase);
                    while (!full[at].passed(phase)) co_await kYield;
                    while (!P[2 * st + (pn & 1)].passed(pn >> 1 & 1u)) co_await kYield;
                    take(at, (int)si, false, shared ? k : 2 * k + st);
                    products[st].push_back({{&empty[at], at}, {&PV[st], -1}});
                    if (k == items - 1) products[st].back().push_back({&O, -1});
                    if (both) empty[at].arrive();
                    ++pn;
                    co_await kYield;
                }
                const int i = k + 2;
                if (i < items) {
                    const int at = (int)ring.at(shared, st, i, true, g.n, phase);
                    while (!full[at].passed(phase)) co_await kYield;
                    take(at, (int)si, true, shared ? i : 2 * i + st);
                    products[st].push_back({{&S[2 * st + (sn & 1)], -1}, {&empty[at], at}});
                    if (both) empty[at].arrive();
                    ++sn;
                    co_await kYield;
                }
            }
            if (items == 0) O.arrive();
            ring.next(shared, g.n);
        }
        products[st].push_back({{nullptr, -1}});
    }

    Process softmax(int st) {
        uint32_t done = 0;
        for (size_t si = 0; si < segs.size(); ++si) {
            const Segment g = segs[si];
            Q.arrive();
            const int items = g.dual || !TWO ? g.n : (g.n - st + 1) / 2;
            for (int k = 0; k < items; ++k) {
                const int buf = 2 * st + (done & 1);
                while (!S[buf].passed(done >> 1 & 1u)) co_await kYield;
                for (int i = pick({0, 0, 0, 3, 40}); i > 0; --i) co_await kYield;
                if (done > 0)
                    while (!PV[st].passed((done - 1u) & 1u)) co_await kYield;
                ++done;
                P[buf].arrive();
                co_await kYield;
            }
            while (!O.passed((uint32_t)si & 1u)) co_await kYield;
        }
    }

public:
    Run(std::vector<Segment> s, uint32_t seed, RingKind k) : rnd(seed), segs(std::move(s)), kind(k) {
        for (int i = 0; i < SLOTS; ++i) {
            full.emplace_back(2);
            empty.emplace_back(kStreams);
            landed.emplace_back(1);
            landed.emplace_back(1);
        }
        for (int i = 0; i < 4; ++i) {
            S.emplace_back(1);
            P.emplace_back(1);
        }
        for (int i = 0; i < 2; ++i) PV.emplace_back(1);
    }
    void operator()() {
        for (int i = 0; i < 4; ++i) procs.push_back(loader(i < 2, i & 1));
        for (int st = 0; st < kStreams; ++st) {
            procs.push_back(mma(st));
            procs.push_back(pipe(st));
            procs.push_back(softmax(st));
        }
        for (size_t i = 0; i < procs.size(); ++i) speed.push_back(pick({1, 1, 5, 30}));
        for (int64_t steps = 0; !procs.empty(); ++steps) {
            const size_t i = rnd() % procs.size();
            if (speed[i] > 1 && rnd() % speed[i]) continue;
            // (a process may add others: it runs outside the list)
            Process p = std::move(procs[i]);
            if (p.step()) procs[i] = std::move(p);
            else {
                procs.erase(procs.begin() + i);
                speed.erase(speed.begin() + i);
            }
            if (rnd() % 500 == 0)
                for (int& x : speed) x = pick({1, 1, 5, 30, 200});
            if (steps > 20000000) wrong("nobody can go on");
        }
        for (const Slot& s : slots)
            if (s.busy) wrong("a slot is left in use");
    }
};

template <int SLOTS, bool TWO, bool Q8>
void run(const std::vector<Segment>& segs, uint32_t seed, RingKind kind) {
    if (kind == kOne) Run<SLOTS, TWO, Q8, OneRing<SLOTS, TWO>>(segs, seed, kind)();
    else Run<SLOTS, TWO, Q8, OwnRing<SLOTS, TWO>>(segs, seed, kind)();
}

}  // namespace

int main(int argc, char** argv) {
    if (argc != 4) return 2;
    const int runs = atoi(argv[1]), seed0 = atoi(argv[2]);
    const RingKind kind = !strcmp(argv[3], "own") ? kOwn : !strcmp(argv[3], "one") ? kOne : kEager;
    int n = 0;
    for (int r = 0; r < runs; ++r) {
        std::mt19937 rnd(seed0 + r);
        const auto segments = [&](bool two) {
            std::vector<Segment> s;
            const int many[] = {1, 1, 2, 3, 4}, tiles[] = {1, 2, 3, 5, 8, 13, 27, 40};
            const int count = many[rnd() % 5];
            for (int i = 0; i < count; ++i) s.push_back({tiles[rnd() % 8], !two || rnd() % 2 == 0});
            return s;
        };
        try {
            const uint32_t seed = 7u * (uint32_t)(seed0 + r);
            // the kernel's slots at head sizes 128 in bf16 and 8 bits, 64, 256 in bf16 and 8 bits
            run<10, true, false>(segments(true), seed, kind);
            run<9, true, true>(segments(true), seed + 1, kind);
            run<20, true, false>(segments(true), seed + 2, kind);
            run<20, true, true>(segments(true), seed + 3, kind);
            run<5, false, false>(segments(false), seed + 4, kind);
            run<4, false, true>(segments(false), seed + 5, kind);
            n += 6;
        } catch (const std::exception& e) {
            printf("run %d: %s\n", r, e.what());
            return 1;
        }
    }
    printf("%d runs\n", n);
    return 0;
}
