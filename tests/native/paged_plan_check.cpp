// Prints the paged attention's shapes and forms (paged_plan.h) for the lines of standard input:
// "s es width rows" as "tokens pitch step joined scratch fixed ctas stages",
// "f B heads kv_heads D room window es" as "cluster tiles workspace_bytes".
#include <cstdio>

#include "paged_plan.h"

int main() {
    char what;
    while (std::scanf(" %c", &what) == 1) {
        if (what == 's') {
            int es, width, rows;
            if (std::scanf("%d %d %d", &es, &width, &rows) != 3) return 1;
            const rowops::PagedShape s = rowops::paged_shape(es, width, rows);
            std::printf("%d %d %d %d %d %d %d %d\n", s.tokens, s.pitch, s.step, s.joined, s.scratch, s.fixed, s.ctas, s.stages);
        } else {
            long long B, heads, kv, D, room, window;
            int es;
            if (std::scanf("%lld %lld %lld %lld %lld %lld %d", &B, &heads, &kv, &D, &room, &window, &es) != 7) return 1;
            const rowops::PagedForm f = rowops::paged_form(B, heads, kv, D, room, window, es);
            std::printf("%d %lld %zu\n", f.cluster, static_cast<long long>(f.tiles),
                        rowops::paged_bytes(B, heads, kv, D, room, window, es));
        }
    }
    return 0;
}
