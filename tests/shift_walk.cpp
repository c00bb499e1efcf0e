// The walk of a shift's workgroups over their items on the CPU, up to as many items as a call may have: each item is
// taken by one workgroup, and every workgroup ends.  Prints "ok".
#include <cstdio>
#include <cstdlib>

#include "kvxfer_ops.h"

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("failed: %s (line %d)\n", #x, __LINE__);      \
            std::exit(1);                                             \
        }                                                             \
    } while (0)

int main()
{
    const int64_t most = 0x7fffffff, grid = KVX_SHIFT_GRID;
    for (int64_t items : {(int64_t)1, grid - 1, grid, grid + 1, 3 * grid + 5, most - grid, most - grid + 1, most - 1, most}) {
        const int64_t workgroups = items < grid ? items : grid;
        int64_t taken = 0;
        for (int64_t b = 0; b < workgroups; ++b) {
            int64_t n = 0;
            for (kvx::ItemWalk w{(uint32_t)b, (uint32_t)workgroups, (uint32_t)items}; w.there(); w.next(), ++n) {
                CHECK((int64_t)w.at == b + n * workgroups && (int64_t)w.at < items && (int32_t)w.at >= 0);
                CHECK(n <= items / workgroups);
            }
            taken += n;
        }
        CHECK(taken == items);
    }
    std::puts("ok");
}
