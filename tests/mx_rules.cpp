// Prints which kernel takes a product with a 4-bit weight; built and asked by
// test_mx_rules_host.py.  Arguments: triples of m, output columns, inner size.
#include <stdio.h>
#include <stdlib.h>
#include "zs_mx_rules.h"

using namespace zs::mx;

int main(int argc, char **argv) {
    for (int i = 1; i + 2 < argc; i += 3) {
        const uint64_t m = strtoull(argv[i], 0, 10), c = strtoull(argv[i + 1], 0, 10);
        const uint64_t inner = strtoull(argv[i + 2], 0, 10);
        const int mx = skinny(m, c) ? 0 : 32 * tile_frags(m, c, kLeastTilesMx);
        const int linear = skinny(m, c) ? 0 : 32 * tile_frags(m, c, kLeastTilesHalf);
        const int grad = m <= kSkinnyM ? 0 : 32 * tile_frags(m, c, kLeastTilesHalf);
        printf("%d %d %d %u\n", mx, linear, grad, grad_parts(m, inner, c));
    }
    return 0;
}
