// Tile kernels on microscaled 4-bit operands.
#include "ffn_tile.cuh"

namespace sat {
namespace ffn {

extern const Variant kScaledTiles[] = {
    //             MX    epilogue CG  BN   P_MN   Q_MN   SWAP   SPLIT
    variant<TileTraits<true, kStore, 2, 256, false, false, false, false>>(),
    variant<TileTraits<true, kGated, 2, 256, false, false, false, false>>(),
    variant<TileTraits<true, kStore, 1, 128, false, false, false, true>>(),
    variant<TileTraits<true, kGated, 1, 256, false, false, false, true>>(),
    variant<TileTraits<true, kStore, 1, 16, false, false, true, true>>(),
    variant<TileTraits<true, kStore, 1, 32, false, false, true, true>>(),
    variant<TileTraits<true, kStore, 1, 64, false, false, true, true>>(),
    variant<TileTraits<true, kGated, 1, 16, false, false, true, true>>(),
    variant<TileTraits<true, kGated, 1, 32, false, false, true, true>>(),
    variant<TileTraits<true, kGated, 1, 64, false, false, true, true>>(),
};
extern const int kNumScaledTiles = sizeof kScaledTiles / sizeof kScaledTiles[0];

}  // namespace ffn
}  // namespace sat
