// Tile kernels of the gated product's backward pass.
#include "ffn_tile.cuh"

namespace sat {
namespace ffn {

extern const Variant kGradTiles[] = {
    //             MX     epilogue CG  BN   P_MN   Q_MN   SWAP   SPLIT
    variant<TileTraits<false, kGrad, 2, 256, false, false, false, false>>(),
    variant<TileTraits<false, kGrad, 2, 256, false, true, false, false>>(),
    variant<TileTraits<false, kGrad, 1, 128, false, false, false, true>>(),
    variant<TileTraits<false, kGrad, 1, 128, false, true, false, true>>(),
    variant<TileTraits<false, kStore, 2, 256, false, false, false, false>>(),
    variant<TileTraits<false, kStore, 2, 256, false, true, false, false>>(),
    variant<TileTraits<false, kStore, 2, 256, true, true, false, false>>(),
    variant<TileTraits<false, kStore, 1, 128, false, false, false, true>>(),
    variant<TileTraits<false, kStore, 1, 128, false, true, false, true>>(),
    variant<TileTraits<false, kStore, 1, 128, true, true, false, true>>(),
};
extern const int kNumGradTiles = sizeof kGradTiles / sizeof kGradTiles[0];

}  // namespace ffn
}  // namespace sat
