// Test program, not part of the library: the stages of the product kernels as state machines on the
// host, with the library's own arithmetic of stages and parities.  Producers load blocks, an issuer
// commits each to the `empty` barrier of every CTA, and every arrival takes a time of its own.  Checks
// that no stage is loaded before its last use is done, and that nothing is still to arrive in a CTA
// when it leaves.
// Usage: stage_ring_check <stages> <blocks> <producers> <ctas> <seed> <last: empty|full>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../block_draft_proposal_gb300/csrc/stage_ring.h"

using dflash2::ring_last_uses;
using dflash2::ring_parity;

struct Barrier {  // one arrival completes a phase; a wait for a parity ends when that phase is over
    uint32_t phase = 0;
    bool passes(uint32_t parity) const { return (phase & 1u) != parity; }
};
struct Producer {
    uint32_t cta, first, next, last;
    bool through = false;
};

int main(int argc, char **argv) {
    if (argc != 7) return 2;
    const uint32_t stages = atoi(argv[1]), blocks = atoi(argv[2]), producers = atoi(argv[3]), ctas = atoi(argv[4]);
    std::mt19937 rng(atoi(argv[5]));
    const bool empties = !strcmp(argv[6], "empty");
    std::vector<std::vector<Barrier>> empty(ctas, std::vector<Barrier>(stages));
    std::vector<Barrier> full(stages);
    std::vector<uint32_t> loads(blocks, 0);
    std::vector<bool> done(blocks, false);
    struct Arrival {
        uint32_t cta, block;
    };
    std::vector<Arrival> on_the_way;
    std::vector<Producer> all;
    for (uint32_t c = 0; c < ctas; ++c)
        for (uint32_t p = 0; p < producers; ++p) {
            // the uses to wait for at the end: of this producer's blocks, every one that is its stage's last
            const uint32_t last = ring_last_uses(p, producers, blocks, stages);
            for (uint32_t k = p; k < blocks; k += producers)
                if ((k + stages >= blocks) != (k >= last)) return printf("last uses of %u: %u\n", p, last), 1;
            all.push_back({c, p, p, last});
        }
    uint32_t issued = 0;
    for (uint32_t idle = 0; idle < 100000; ++idle) {
        bool left = issued == blocks && on_the_way.empty();
        for (auto &p : all) left = left && p.through;
        if (left) return 0;
        // a CTA leaves when its producers are through and the sums of all blocks have been read
        for (uint32_t c = 0; c < ctas && issued == blocks; ++c) {
            bool through = true;
            for (auto &p : all) through = through && (p.cta != c || p.through);
            for (auto &a : on_the_way)
                if (through && a.cta == c) return printf("block %u arrives in a CTA that left\n", a.block), 1;
        }
        const uint32_t pick = rng() % (uint32_t)(all.size() + 2);
        if (pick < all.size()) {
            Producer &p = all[pick];
            if (p.through) continue;
            if (p.next < blocks) {  // load the next block
                const uint32_t k = p.next, s = k % stages;
                if (!empty[p.cta][s].passes(ring_parity(k, stages) ^ 1u)) continue;
                if (k >= stages && !done[k - stages]) return printf("block %u loaded over block %u\n", k, k - stages), 1;
                if (++loads[k] == ctas) ++full[s].phase;  // all of it has landed
                p.next += producers;
            } else if (p.last < blocks) {  // the end: wait for a last use
                const uint32_t s = p.last % stages, parity = ring_parity(p.last, stages);
                if (!(empties ? empty[p.cta][s] : full[s]).passes(parity)) continue;
                p.last += producers;
            } else {
                p.through = true;
            }
        } else if (pick == all.size()) {  // the MMAs of the next block, and their commit
            if (issued < blocks && full[issued % stages].passes(ring_parity(issued, stages))) {
                done[issued] = true;
                for (uint32_t c = 0; c < ctas; ++c) on_the_way.push_back({c, issued});
                ++issued;
            }
        } else if (!on_the_way.empty()) {  // an arrival; those of one CTA come in order
            const size_t i = rng() % on_the_way.size();
            size_t j = 0;
            while (on_the_way[j].cta != on_the_way[i].cta) ++j;
            ++empty[on_the_way[j].cta][on_the_way[j].block % stages].phase;
            on_the_way.erase(on_the_way.begin() + (long)j);
        }
    }
    return printf("no end\n"), 1;
}
