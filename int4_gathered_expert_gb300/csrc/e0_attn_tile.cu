// Instances of the tile kernels (e0_attn_tile.cuh).
#include "e0_attn_tile.cuh"

namespace e0 {

size_t attn_tile_ws_bytes(int B, int max_q, int G, int D) { return tile_ws_bytes(B, max_q, G, D); }

bool attn_tile_merges(const AttnArgs& a) {
    return a.window == 0 && tile_jobs(a.B, a.max_q, a.Hq / a.Hkv, a.D) * a.Hkv <= tile_blocks();
}

int attn_tile(const AttnArgs& a, const TilePrefix* prefix, int dtype, void* ws, cudaStream_t s) {
    const TileArgs t = tile_args(a, prefix, dtype, ws);
    return a.D == 64 ? tile_launch_d<64>(t, dtype, s) : a.D == 128 ? tile_launch_d<128>(t, dtype, s) : tile_launch_d<256>(t, dtype, s);
}

}  // namespace e0
