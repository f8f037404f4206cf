// Tile kernels on 16-bit operands.
#include "ffn_tile.cuh"

namespace sat {
namespace ffn {

extern const Variant kHalfTiles[] = {
    //             MX     epilogue CG  BN   P_MN   Q_MN   SWAP   SPLIT
    variant<TileTraits<false, kGated, 2, 256, false, false, false, false>>(),
    variant<TileTraits<false, kGated, 2, 256, false, true, false, false>>(),
    variant<TileTraits<false, kGated, 1, 128, false, false, false, true>>(),
    variant<TileTraits<false, kGated, 1, 128, false, true, false, true>>(),
    variant<TileTraits<false, kGated, 1, 16, false, false, true, true>>(),
    variant<TileTraits<false, kGated, 1, 32, false, false, true, true>>(),
    variant<TileTraits<false, kGated, 1, 64, false, false, true, true>>(),
    variant<TileTraits<false, kGated, 1, 16, true, false, true, true>>(),
    variant<TileTraits<false, kGated, 1, 32, true, false, true, true>>(),
    variant<TileTraits<false, kGated, 1, 64, true, false, true, true>>(),
};
extern const int kNumHalfTiles = sizeof kHalfTiles / sizeof kHalfTiles[0];

}  // namespace ffn
}  // namespace sat
