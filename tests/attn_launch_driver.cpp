// For each call "B T nseq packed Hk Hv dk dv" on stdin: whether its workgroups can be numbered, and the most that one of linear
// attention's launches has.
#include <algorithm>
#include <cstdint>
#include <iostream>

#include "../gated_delta_rule_70_amd/csrc/layer_plan.hpp"

using namespace gdr;

namespace {
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
// a sweep of `roles` over db columns of units' heads, narrow or not
int64_t sweep(int64_t units, int64_t Hk, int64_t Hv, int64_t roles, int64_t db, bool narrow) {
    const int tiles = narrow ? attn_tiles(db, units * Hv * roles * attn_slices(db)) : attn_tiles(db);
    return up(units * Hk, 8) * 8 * roles * attn_slices(db, tiles) * (Hv / Hk);
}
}  // namespace

int main() {
    int64_t B, T, nseq, packed, Hk, Hv, dk, dv;
    while (std::cin >> B >> T >> nseq >> packed >> Hk >> Hv >> dk >> dv) {
        int64_t most = nseq * Hv * (dv / 32);  // a step of as many sequences
        auto see = [&](int64_t blocks) { most = std::max(most, blocks); };
        const int64_t elems = dk * dv / 1024;
        const AttnPlan f = attn_plan(T, nseq, Hv * attn_slices(dv), packed != 0, false), b = attn_plan(T, nseq, Hv, packed != 0, true);
        if (f.seg) {
            see(sweep(f.slots - nseq, Hk, Hv, 1, dv, true));
            see((f.slots - nseq) * Hv * elems);
        }
        see(sweep(f.slots, Hk, Hv, 1, dv, true));
        if (b.seg) {
            see(sweep(b.slots, Hk, Hv, 2, dv, true));
            see(nseq * Hv * elems);
        }
        see(sweep(b.slots, Hk, Hv, 3, dk, false));
        see(sweep(b.slots, Hk, Hv, 1, dv, true));
        see(b.slots * Hv);
        if (Hk < Hv) see(up(2 * B * Hk * T * dk, 1024));
        std::cout << attn_numbered(nseq, B, T, Hv) << " " << most << std::endl;
    }
}
