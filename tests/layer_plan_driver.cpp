// Prints how the layer operators lay out the calls given on stdin, one a line:
//   scan T D nseq packed es     -> chunk units ntile
//   ffn M D F es                -> the forward's, dx's and the weights' kernels
//   ce N D V es                 -> the forward's kernel, then per kind of piece: width, dl's, dW's and dx's
// A kernel is "any", "rows<mt>x<nt>" or "<tile>", with "/<slices>" where k is cut.
#include <iostream>
#include <string>

#include "../gated_delta_rule_70_amd/csrc/layer_plan.hpp"

using namespace gdr;

static std::string name(const GemmOp &o, int es, int NB, bool both, bool whole) {
    const Path p = path_of(o, es, NB, both, whole);
    if (p.kind == Path::kAny) return "any";
    if (p.kind == Path::kRows) return "rows" + std::to_string(p.mt) + "x" + std::to_string(p.nt);
    return std::to_string(p.tile);
}
static std::string stored(GemmOp o, int es) {
    const Choice c = store_choice(o, es);
    o.tile = c.tile;
    const std::string n = name(o, es, 1, false, true);
    return c.slices > 1 ? n + "/" + std::to_string(c.slices) : n;
}

int main() {
    std::string what;
    while (std::cin >> what) {
        int64_t a, b, c, es;
        if (what == "scan") {
            int64_t packed;
            std::cin >> a >> b >> c >> packed >> es;
            const ScanPlan p = scan_plan(a, b, c, packed != 0, scan_vec(b, (int)es));
            std::cout << p.chunk << " " << p.units << " " << p.ntile << "\n";
            continue;
        }
        std::cin >> a >> b >> c >> es;
        const int e = (int)es;
        if (what == "ffn") {
            std::cout << name(ffn_fwd_product(a, b, c), e, 2, true, true) << " " << stored(ffn_dx_product(a, b, c), e) << " "
                      << stored(ffn_dw_product(a, b, c), e) << "\n";
            continue;
        }
        std::cout << name(ce_logits_product(a, b, c), e, 1, true, false);
        const int64_t piece = ce_piece(a, c);
        int64_t last = 0;
        for (int64_t v = 0; v < c; v += piece) {
            const int64_t width = c - v < piece ? c - v : piece;
            if (width != last)
                std::cout << " " << width << " " << name(ce_logits_product(a, b, width), e, 1, true, true) << " "
                          << stored(ce_dw_product(a, b, piece, width), e) << " " << stored(ce_dx_product(a, b, piece, width), e);
            last = width;
        }
        std::cout << "\n";
    }
    return 0;
}
