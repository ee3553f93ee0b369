// The kernel and tile of each call named on the standard input (q8_mx_plan.h), compiled for the
// host.  A line: format, rows, projections, 1 where rows are quantised on their way out, tokens.
// Answers: "narrow", "columns R" or "wide RT", and the number of tiles.
#include <cstdio>

#include "q8_mx_plan.h"

int main() {
    int form, projections, quantised;
    long long rows, live;
    while (std::scanf("%d %lld %d %d %lld", &form, &rows, &projections, &quantised, &live) == 5) {
        const q8::MxPlan p = q8::mx_plan(form, rows, projections == 2, quantised != 0, live);
        if (p.way == q8::MxPlan::kNarrow) {
            std::printf("narrow 0 0\n");
            continue;
        }
        const bool wide = p.way == q8::MxPlan::kWide;
        const long long tile = (wide ? 256 : 32 * p.tile) / projections, tokens = wide ? 64 * p.tile : 64;
        std::printf("%s %d %lld\n", wide ? "wide" : "columns", p.tile, (rows + tile - 1) / tile * ((live + tokens - 1) / tokens));
    }
    return 0;
}
