// Arrays of three strides on the CPU: those taken as having no two elements in one place have none, and every order of
// dimensions that lie one within the other is taken.  Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kvxfer_opshost.h"

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("failed: %s (line %d)\n", #x, __LINE__);      \
            std::exit(1);                                             \
        }                                                             \
    } while (0)

int main()
{
    int64_t taken = 0, refused = 0;
    for (int64_t n = 1; n <= 3; ++n)
        for (int32_t heads = 1; heads <= 3; ++heads)
            for (int64_t layers = 1; layers <= 3; ++layers)
                for (int64_t token = 0; token <= 12; ++token)
                    for (int64_t head = 0; head <= 12; ++head)
                        for (int64_t layer = 0; layer <= 12; ++layer) {
                            const int32_t dim = 2;
                            std::vector<int> seen(2 * 12 * 3 + dim, 0);
                            int most = 0;
                            for (int64_t a = 0; a < n; ++a)
                                for (int64_t b = 0; b < heads; ++b)
                                    for (int64_t c = 0; c < layers; ++c)
                                        for (int32_t d = 0; d < dim; ++d) {
                                            int &at = seen[a * token + b * head + c * layer + d];
                                            most = std::max(most, ++at);
                                        }
                            const bool ok = kvx::apart(n, heads, token, head, dim, layers, layer);
                            CHECK(!ok || most == 1);
                            (ok ? taken : refused) += 1;
                            // two dimensions, as attention's results are checked
                            if (layers == 1) CHECK(kvx::apart(n, heads, token, head, dim) == ok);
                        }
    CHECK(taken > 0 && refused > 0);
    const int64_t sizes[3] = {5, 3, 4};  // tokens, heads, layers
    int order[3] = {0, 1, 2};
    do {
        int64_t stride[3], span = 8;
        for (int i : order) stride[i] = span, span *= sizes[i];
        CHECK(kvx::apart(sizes[0], (int32_t)sizes[1], stride[0], stride[1], 8, sizes[2], stride[2]));
        for (int i = 0; i < 3; ++i) {
            int64_t less[3] = {stride[0], stride[1], stride[2]};
            less[i] -= 1;
            CHECK(!kvx::apart(sizes[0], (int32_t)sizes[1], less[0], less[1], 8, sizes[2], less[2]));
        }
    } while (std::next_permutation(order, order + 3));
    std::puts("ok");
}
