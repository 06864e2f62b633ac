// The rings of the norm and the recurrence, played through on the host: the copies
// that are in flight when a wait gives up, and those that drain_ring waits for.
#include <cstdio>
#include <set>

#include "ring.h"

// The copies of tiles 0, 1, ... go into the slots in turn, a phase of the slot's
// barrier each.
static int slot_of(int tile, int stages) { return tile % stages; }
static unsigned phase_of(int tile, int stages) { return unsigned(tile / stages) & 1u; }

// One group over `tiles` tiles whose wait for tile `fails` gives up.  late_refill: a
// slot is filled anew one tile after it was read (the norm's backward pass), else
// behind the tile itself.
static bool play(int stages, int tiles, int fails, bool late_refill) {
    std::set<int> flying;  // issued and not waited for
    const auto issue = [&](int tile) {
        if (tile < tiles) flying.insert(tile);
    };
    for (int k = 0; k < stages; ++k) issue(k);
    int slot = 0, used = -1;
    unsigned parity = 0;
    for (int r = 0; r < tiles; ++r) {
        if (slot != slot_of(r, stages) || parity != phase_of(r, stages)) return false;
        if (r == fails) {
            std::set<int> waited;
            mss::drain_ring(slot, parity, stages, late_refill && used >= 0 ? stages - 1 : stages, [&](int k, int at, uint32_t phase) {
                if (r + k < tiles && at == slot_of(r + k, stages) && phase == phase_of(r + k, stages)) waited.insert(r + k);
            });
            return waited == flying;
        }
        flying.erase(r);
        if (late_refill) {
            if (used >= 0) issue(r + stages - 1);
            used = slot;
        } else {
            issue(r + stages);
        }
        if (++slot == stages) slot = 0, parity ^= 1;
    }
    return false;
}

int main() {
    for (int late = 0; late < 2; ++late)
        for (int stages = late ? 2 : 1; stages <= 4; ++stages)
            for (int tiles = 1; tiles <= 13; ++tiles)
                for (int fails = 0; fails < tiles; ++fails)
                    if (!play(stages, tiles, fails, late != 0)) {
                        std::printf("%d stages, %d tiles, tile %d gives up, %s\n", stages, tiles, fails, late ? "late refill" : "refill at once");
                        return 1;
                    }
    std::puts("ok");
}
