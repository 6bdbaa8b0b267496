// Checks how a block whose waits gave up leaves its ring of slots (f8_ring.h),
// against a model of the slots' mbarriers: a phase ends when its copy lands, a
// wait for a parity returns once the phase of that parity is over, and a second
// copy into a slot whose phase is not over is an error.  A thread fills the
// slots ahead of its items and refills them as the items arrive, up to a wait
// that gives up, with any of the copies then under way landed or not; or one
// thread issues all copies and is done before another's wait for one gives up.
// Afterwards every copy must have landed, and no wait may name a phase that is
// not the slot's own (it would return at once, or never).
// Usage: ring_check [cases]; prints "<n> cases, <m> mismatches".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../float8_mixed_precision_gb300/csrc/f8_ring.h"

struct Slot {
    int64_t over = 0;       // phases that have ended
    bool under_way = false; // the copy of phase `over` has been issued and not landed
};

struct Model {
    std::vector<Slot> slots;
    int64_t bad = 0;

    explicit Model(int n) : slots(n) {}
    void issue(int64_t seq)
    {
        Slot &s = slots[seq % slots.size()];
        if (s.under_way || s.over != seq / static_cast<int64_t>(slots.size()))
            ++bad;
        s.under_way = true;
    }
    void land(int i)
    {
        if (slots[i].under_way) {
            slots[i].under_way = false;
            ++slots[i].over;
        }
    }
    // A wait with the given parity: returns at once if the phase before the
    // current one has it, else when the current one ends.
    void wait(int i, uint32_t parity)
    {
        Slot &s = slots[i];
        const bool current = (s.over & 1) == parity;
        if (s.under_way && !current)
            ++bad;  // returns while the copy is under way
        if (!s.under_way && current)
            ++bad;  // no copy ends this phase: runs into the limit
        if (current)
            land(i);
    }
    int64_t left() const
    {
        int64_t n = 0;
        for (const Slot &s : slots)
            n += s.under_way;
        return n;
    }
};

static uint32_t rnd()
{
    static uint64_t x = 88172645463325252ull;
    x ^= x << 13, x ^= x >> 7, x ^= x << 17;
    return static_cast<uint32_t>(x >> 11);
}

// `count` items over `slots` slots; the wait for item `at` gives up (at ==
// count: none does).
static int64_t taking(int slots, int64_t count, int64_t at)
{
    Model m(slots);
    uint32_t issued = 0;
    for (int64_t i = 0; i < slots && i < count; ++i)
        m.issue(issued++);
    bool ok = true;
    for (int64_t i = 0; i < count; ++i) {
        if (ok && i == at) {
            // the copies behind this one may have landed; it may do so late
            for (int64_t j = i + (rnd() & 1 ? 0 : 1); j < i + slots && j < count; ++j)
                if (rnd() & 1)
                    m.land(f8::ring_slot(j, slots));
            ok = false;
        }
        if (ok) {
            m.wait(f8::ring_slot(i, slots), f8::ring_parity(i, slots));
            if (i + slots < count)
                m.issue(issued++);
        }
    }
    if (!ok)
        f8::ring_drain(issued, slots, [&](int slot, uint32_t parity) { m.wait(slot, parity); });
    return m.bad + m.left();
}

// The thread that issues the copies is not the one that takes them: it has issued
// the last of `count` while the taker has yet to give up, so it waits for them
// whether or not anyone has.
static int64_t apart(int slots, int64_t count)
{
    Model m(slots);
    uint32_t issued = 0;
    int64_t taken = 0;
    while (issued < count) {
        if (issued < taken + slots && (rnd() & 1))
            m.issue(issued++);
        else if (taken < issued)
            m.wait(f8::ring_slot(taken, slots), f8::ring_parity(taken, slots)), ++taken;
    }
    for (int i = 0; i < slots; ++i)
        if (rnd() & 1)
            m.land(i);
    f8::ring_drain(issued, slots, [&](int slot, uint32_t parity) { m.wait(slot, parity); });
    return m.bad + m.left();
}

int main(int argc, char **argv)
{
    const long cases = argc > 1 ? atol(argv[1]) : 2000;
    long n = 0, bad = 0;
    for (int slots = 1; slots <= 8; ++slots)
        for (int64_t count = 0; count <= 30; ++count)
            for (int64_t at = 0; at <= count; ++at, ++n)
                bad += taking(slots, count, at) != 0;
    for (long i = 0; i < cases; ++i, ++n) {
        const int64_t count = 1 + rnd() % 2000;
        bad += taking(1 + rnd() % 8, count, rnd() % (count + 1)) != 0;
        bad += apart(1 + rnd() % 8, count) != 0;
    }
    printf("%ld cases, %ld mismatches\n", n, bad);
    return bad != 0;
}
