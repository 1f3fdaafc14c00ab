// Attention of one new token over a paged key-value cache: arguments and launchers (internal to
// libgdr2).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr2 {

struct Cache {  // [pages][page][Hkv][D] with any strides (elements) between pages, tokens and heads
    void *k, *v;
    long long ks[3], vs[3];  // page, token, head
    const int* table;        // [B][max_pages]
    int pages, page, shift, max_pages;
};

struct AttnArgs {
    const void* q;       // [B][Hq][D]
    Cache c;
    const int* lengths;  // [B]: tokens a sequence holds
    void* o;             // [B][Hq][D]
    float* lse;          // [B][Hq] or null
    float* part;         // workspace: partial results, 2 a workgroup
    int B, Hq, Hkv, D, G;  // G = Hq / Hkv query heads share a key head
    int gh, NG;            // heads of a head group (at most 16), groups of a key head
    int window;            // 0: all tokens
    float scale2;          // scale * log2(e)
    int wgs;               // workgroups that share the tokens
};

struct AppendArgs {
    const void *k, *v;   // [tokens][Hkv][D]
    Cache c;
    const int* starts;   // [B]: tokens a sequence holds before the call
    const int* cu;       // [B + 1] or null: one token a sequence
    int B, tokens, Hkv, D;
};

constexpr int ATTN_WGS = 256;  // one workgroup of eight waves on each of the 256 compute units
constexpr int ATTN_COST = 6;   // of a row, in units: its own loads and its waves' join

// Tokens of a unit, the piece that a wave takes at a time, and the units that a row has at most, by its table
// or its window (which may begin inside a unit).
constexpr int attn_unit_tokens(bool bf16) { return bf16 ? 32 : 16; }
inline long long attn_max_units(const Cache& c, int window, int unit) {
    long long tokens = (long long)c.max_pages << c.shift;
    if (window > 0 && window < tokens) tokens = (long long)window + unit;
    return (tokens + unit - 1) / unit;
}
// The most places that the line of all rows can have (gdr2_attn.hip); an empty row has a unit too.
inline long long attn_line_places(const AttnArgs& a, int unit) {
    const long long units = attn_max_units(a.c, a.window, unit);
    return (long long)a.B * a.Hkv * a.NG * ((units > 0 ? units : 1) + ATTN_COST);
}

// floats of one partial result: gh rows of D sums, then their maxima and weights (padded to 16 bytes)
inline size_t attn_part_floats(int gh, int D) { return (size_t)gh * (D + 4); }

hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_append(const AppendArgs& a, bool bf16, hipStream_t stream);

}  // namespace gdr2
