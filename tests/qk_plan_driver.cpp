// Prints how the norms of queries and keys lay out the calls given on stdin, one "B T Hq Hk d" a line: tokens of a workgroup's
// tile, tiles, steps of all heads of a tile, steps of a workgroup's turn, workgroups of the backward.
#include <cstdint>
#include <iostream>

#include "../gated_delta_rule_70_amd/csrc/layer_plan.hpp"

using namespace gdr;

int main() {
    int64_t B, T, Hq, Hk, d;
    while (std::cin >> B >> T >> Hq >> Hk >> d) {
        int lanes = 2;
        while (8 * lanes < d) lanes *= 2;
        const int64_t rows = B * T;
        const int tokens = qk_tokens(rows, Hq + Hk, 256 / lanes) > 4 ? (lanes < 32 ? 16 : 8) : 4, heads = 256 / lanes / tokens;
        const int64_t tiles = (rows + tokens - 1) / tokens, all = (Hq + heads - 1) / heads + (Hk + heads - 1) / heads, steps = qk_steps(tiles, all);
        std::cout << tokens << " " << tiles << " " << all << " " << steps << " " << qk_groups(tiles * ((all + steps - 1) / steps)) << std::endl;
    }
}
