// zs_mx_rules.h -- which kernel takes a product with a 4-bit weight, by its
// sizes.  Host only, and free of HIP, so that a host program can ask.
#ifndef ZS_MX_RULES_H
#define ZS_MX_RULES_H

#include <stdint.h>

namespace zs {
namespace mx {

constexpr uint32_t kSkinnyWaves = 8; // of a workgroup of the kernels for few rows
constexpr uint64_t kSkinnyM = 64;    // the most rows they take
constexpr uint32_t kGradCols = 64;   // columns of a workgroup of the gradient's
constexpr uint32_t grad_waves(int mt) { return mt == 1 ? 16 : 8; }

// Tiles of a tiled product: 256 x 256 if they take more than half of the
// chip's 256 CUs (one of them a CU), else 128 x 128 if there are `least` of
// those (two a CU), else 64 x 64.  Measured at K = 4096, N = 4096, bfloat16
// linear: 2048 rows (128 tiles of 256, 512 of 128) 103 us against 87; 2047 x
// 6400 x 1600 (200 and 800) 49 against 65; 512 rows (128 of 128, 512 of 64)
// 69 against 43.  In 4 bits a step has half the loads and no decoding, and
// 128 x 128 pays earlier: 512 rows 18 us against 25.
constexpr uint64_t kCUs = 256;
constexpr uint64_t kLeastTilesMx = kCUs / 4, kLeastTilesHalf = kCUs;
inline uint64_t tiles_of(uint64_t M, uint64_t C, uint64_t tile) {
    return (M + tile - 1) / tile * ((C + tile - 1) / tile);
}
inline int tile_frags(uint64_t M, uint64_t C, uint64_t least) {
    return tiles_of(M, C, 256) > kCUs / 2 ? 8 : tiles_of(M, C, 128) >= least ? 4 : 2;
}

// Whether the skinny kernels take a product: 17 and more rows make each of
// their workgroups read much of the left operand, and from 33 rows on 64 x 64
// tiles are faster if they fill half the chip (64 rows, K = 4096: N = 4096 19
// us against 28 tiled, N = 11008 51 against 29).
inline bool skinny(uint64_t M, uint64_t N) {
    return M <= kSkinnyM / 2 || (M <= kSkinnyM && tiles_of(M, N, 64) < kCUs / 2);
}

// Whether the kernel that holds the left operand in registers takes a
// product: `most` steps a wave hold K.
inline bool in_registers(uint64_t nb, uint32_t most) {
    return nb >= 8 && nb <= 4ull * kSkinnyWaves * most;
}

// Parts of the sum over the weight's rows.  The kernel for few rows gets a
// workgroup for each CU, each wave a unit of 32 rows at least (two a CU read
// more of dy and join more: 64 x 50257 x 1600 77 us against 68, four 90); whole
// sums took 525 us there, 153 for 1 x 50257 x 1600 (30 now).
// The tiled kernels run two workgroups a CU, of 256 x 256 tiles one.  A part is
// worth its partial sums and the join where it holds enough steps of 64 rows
// (m x n x k, bfloat16, whole against in parts):
// - 64 x 64: 16 for up to 128 tiles (65 x 50257 x 1600 548 us against 78; 65 x
//   2048 x 4096 20 and 17), 32 for more (512 x 2048 x 1600 20.8 against 25.4 in
//   two parts, 512 x 4096 x 1600 47 and 36);
// - 128 x 128: 48 (2048 x 4096 x 2048 54 and 60, 2048 x 6144 x 2048 80 and 80,
//   2048 x 32000 x 2048 381 and 328);
// - 256 x 256: three parts of up to 170 tiles take two thirds of a round: 48
//   (4352 x 4096 x 2048 122 and 129, 4352 x 11008 x 2048 298 and 250).  Two parts
//   are two half rounds, as long as one, and cost 50-60 us more (4096 x 4096 x
//   4096 123 and 175): only the fp32 sums of 768 steps and more are halved, for
//   3-4% (4096 x 50257 x 4096 1661 and 1726).
// The join takes a grid of at most 65,535 rows.
inline uint32_t grad_parts(uint64_t m, uint64_t N, uint64_t K) {
    if (m > 65535)
        return 1;
    uint64_t want, most;
    if (m <= kSkinnyM) {
        want = kCUs / ((K + kGradCols - 1) / kGradCols);
        most = (N + 31) / 32 / (m <= 16 ? grad_waves(1) : grad_waves(4));
    } else {
        const int frags = tile_frags(m, K, kLeastTilesHalf);
        const uint64_t tiles = tiles_of(m, K, 32 * frags), steps = (N + 63) / 64;
        want = 2 * kCUs / tiles;
        most = steps / (frags == 2 ? (tiles > kCUs / 2 ? 32 : 16)
                        : frags == 4 || want == 3 ? 48
                                                  : 384);
        if (frags == 8 && most < want) // all of them or none
            most = 1;
    }
    const uint64_t parts = want < most ? want : most;
    return parts < 2 ? 1 : (uint32_t)parts;
}

} // namespace mx
} // namespace zs

#endif
