// Drafted tokens over a paged key-value cache: arguments, sizes and launchers (internal to libgdr2).
#pragma once
#include "gdr2_attn.hpp"

namespace gdr2 {

constexpr int TREE_MAX = 64;  // drafts of a row at most: a draft's ancestors are bits of one 64-bit number

struct TreeArgs {
    const void* q;        // [B][T][Hq][D]
    const int* parents;   // [B][T]
    Cache c;
    const int* starts;    // [B]: tokens a sequence holds, its drafts behind them
    void* o;              // [B][T][Hq][D]
    float* lse;           // [B][T][Hq] or null
    float* part;          // workspace: partial results, 2 a workgroup
    int B, T, Hq, Hkv, D, G;
    int window;           // 0: all tokens
    float scale2;         // scale * log2(e)
    int nc, rg, nb;       // 16-row column tiles a wave, waves side by side, blocks of 16 nc rg rows a key head
    int wide, neg;        // wide: rows on tiles in LDS, scale2 not negative or zero: neg turns q's sign
    int unit, cost;       // tokens of a unit; of a row, in units: its own loads and its join
    int wgs, share_min;   // workgroups that share the line of rows, places one takes at least
};

struct KeepArgs {
    Cache c;
    const int *starts, *path;  // [B], [B][P]
    int* lengths;              // [B] or null
    int B, P, Hkv, D, es;
};

// Four waves of rows side by side: tiles of 64 tokens where the tables leave a workgroup few of them, us with 64 and 128:
// 1 sequence of 777 tokens, 12 drafts, 16 heads over 2 16.6 and 19.1; 32 of 200 to 16384, 32 drafts, 32 over 8 138 and 122.
inline int tree_tile(const TreeArgs& a) {
    const long long tiles = (((long long)a.c.max_pages << a.c.shift) + 63) / 64;
    return tiles * a.B * a.Hkv * a.nb <= 4 * a.wgs ? 64 : 128;
}

// How the T G rows of a key head are laid out over waves and workgroups. Up to 32 of them, and fp32: waves that take 16 or
// 32 rows against units straight from the cache (gdr2_tree.hip). More, in bf16: waves of 32 rows side by side on tiles in
// LDS (gdr2_tree_wide.hip).
inline void tree_rows(TreeArgs& a, bool bf16) {
    const int rows = a.T * a.G;
    a.wgs = ATTN_WGS;
    a.wide = bf16 && rows > 32;
    a.nc = rows > 16 ? 2 : 1;
    a.rg = a.wide ? 2 : 1;
    const int tiles = (rows + 16 * a.nc - 1) / (16 * a.nc);
    while (a.rg < 8 && a.rg < tiles) a.rg *= 2;
    a.nb = (tiles + a.rg - 1) / a.rg;
    // tiles of 128 tokens, two blocks of 32 a wave, where LDS and the work are there for them (measured at tree_tile)
    a.unit = !a.wide ? attn_unit_tokens(bf16) : a.rg == 2 || (a.rg == 4 && tree_tile(a) == 128) ? 128 : 64;
    // (wide, us with 1, 3 and 6 places a row: 32 ragged trees of 32 drafts 133, 119, 124; 8 of 2000 tokens 34.7, 32.4, 34.0; 200 of
    // 700, 12 drafts 54.6, 56.1, 56.9. With 1, 2 and 5 places a workgroup at least: 1 of 777, 12 drafts 16.7, 15.7, 19.7; 1 of
    // 4096, 32 drafts 28.5, 28.5, 27.2)
    a.cost = a.wide ? 3 : ATTN_COST;
    a.share_min = a.wide ? 2 : a.cost + 8 / a.rg;
}
inline size_t tree_part_floats(const TreeArgs& a) { return (size_t)16 * a.nc * a.rg * (a.D + 4); }
// behind the parts: four numbers a workgroup (gdr2_tree_wide.hip)
__host__ __device__ inline int* tree_heads(const TreeArgs& a) {
    return (int*)(a.part + 2 * (size_t)a.wgs * (16 * a.nc * a.rg * (a.D + 4)));
}
inline size_t tree_workspace(const TreeArgs& a) {
    return 2 * (size_t)a.wgs * tree_part_floats(a) * sizeof(float) + (a.wide ? 16 * (size_t)a.wgs : 0);
}
inline long long tree_max_units(const TreeArgs& a) {
    long long tokens = (long long)a.c.max_pages << a.c.shift;
    if (a.window > 0 && (long long)a.window + a.T < tokens) tokens = (long long)a.window + a.T + a.unit;
    return (tokens + a.unit - 1) / a.unit;
}
inline long long tree_line_places(const TreeArgs& a) {
    const long long units = tree_max_units(a);
    return (long long)a.B * a.Hkv * a.nb * ((units > 0 ? units : 1) + a.cost);
}

hipError_t launch_tree_wide(const TreeArgs& a, hipStream_t stream);
hipError_t launch_tree(const TreeArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_keep(const KeepArgs& a, hipStream_t stream);

}  // namespace gdr2
