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
    int wgs, share_min;   // workgroups that share the line of rows, places one takes at least
};

struct KeepArgs {
    Cache c;
    const int *starts, *path;  // [B], [B][P]
    int* lengths;              // [B] or null
    int B, P, Hkv, D, es;
};

// how the T G rows of a key head are laid out over waves and workgroups
inline void tree_rows(TreeArgs& a) {
    const int rows = a.T * a.G;
    a.nc = rows > 16 ? 2 : 1;
    const int tiles = (rows + 16 * a.nc - 1) / (16 * a.nc);
    a.rg = 1;
    while (a.rg < 8 && a.rg < tiles) a.rg *= 2;
    a.nb = (tiles + a.rg - 1) / a.rg;
    a.wgs = ATTN_WGS;
    a.share_min = ATTN_COST + 8 / a.rg;
}
inline size_t tree_part_floats(const TreeArgs& a) { return (size_t)16 * a.nc * a.rg * (a.D + 4); }
inline long long tree_max_units(const TreeArgs& a, int unit) {
    long long tokens = (long long)a.c.max_pages << a.c.shift;
    if (a.window > 0 && (long long)a.window + a.T < tokens) tokens = (long long)a.window + a.T + unit;
    return (tokens + unit - 1) / unit;
}
inline long long tree_line_places(const TreeArgs& a, int unit) {
    const long long units = tree_max_units(a, unit);
    return (long long)a.B * a.Hkv * a.nb * ((units > 0 ? units : 1) + ATTN_COST);
}

hipError_t launch_tree(const TreeArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_keep(const KeepArgs& a, hipStream_t stream);

}  // namespace gdr2
