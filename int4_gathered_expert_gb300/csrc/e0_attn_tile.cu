// Instances of the tile kernels (e0_attn_tile.cuh).
#include "e0_attn_tile.cuh"

namespace e0 {

size_t attn_tile_ws_bytes(int B, int max_q, int G, int D) { return tile_ws_bytes(B, max_q, G, D); }

int attn_tile(const AttnArgs& a, int dtype, void* ws, cudaStream_t s) {
    const TileArgs t = tile_args(a, dtype, ws);
    return a.D == 64 ? tile_launch_d<64>(t, dtype, s) : a.D == 128 ? tile_launch_d<128>(t, dtype, s) : tile_launch_d<256>(t, dtype, s);
}

}  // namespace e0
