// Device building blocks of attention over a paged key-value cache: a unit of its tokens in registers.
#pragma once
#include "gdr2_attn.hpp"
#include "gdr2_device.hpp"

namespace gdr2 {

template <class OT>
constexpr int attn_unit() { return attn_unit_tokens(sizeof(OT) == 2); }
constexpr int AW = 8;           // waves of a workgroup

// One unit's keys and values in registers, as loaded.
template <class OT, int D>
struct AttnTile;
template <int D>
struct AttnTile<bf16, D> {
    static constexpr int EV = D / 16;
    typedef bf16 VT __attribute__((ext_vector_type(EV)));
    bf16x8 k[2][D / 32];  // [token tile][channel block]
    VT v[8];              // token 16 (e / 4) + 4 lq + e % 4, channels EV li ..
    int ok;               // bit s: token tile s lies on a valid page
};
template <int D>
struct AttnTile<float, D> {
    static constexpr int EV = D / 16;
    f32x4 k[D / 16];      // channels 16 s + 4 lq ..
    f32x4 v[4][EV / 4];   // token 4 lq + i
    int ok;
};

// The pages of unit u of sequence b, by token tile: negative where there is none, or past the tokens held.
template <class OT>
__device__ __forceinline__ void attn_pages(const Cache& c, int b, int u, int hi, bool any, int (&pg)[2]) {
    constexpr int U = attn_unit<OT>();
#pragma unroll
    for (int s = 0; s < U / 16; ++s) {
        const int tok = u * U + 16 * s;
        pg[s] = -1;
        if (any && tok < hi) {
            const int p = c.table[(size_t)b * c.max_pages + (tok >> c.shift)];
            pg[s] = (unsigned)p < (unsigned)c.pages ? p : -1;
        }
    }
}

// pg[s]: page of token tile s of the unit, or negative. Tiles never straddle pages (a page holds a
// multiple of 16 tokens). Invalid tiles read page 0 and are masked.
template <class OT, int D>
__device__ __forceinline__ void attn_ok(const int (&pg)[2], AttnTile<OT, D>& t) {
    t.ok = 0;
#pragma unroll
    for (int s = 0; s < attn_unit<OT>() / 16; ++s)
        if (pg[s] >= 0) t.ok |= 1 << s;
}
// token tile s of the unit
template <class OT, int D>
__device__ __forceinline__ void attn_load_k(const Cache& c, int u, int hkv, const int (&pg)[2], int s, AttnTile<OT, D>& t) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const int tok = (u * attn_unit<OT>() + 16 * s) & (c.page - 1);
    const long long page = pg[s] >= 0 ? pg[s] : 0;
    const OT* kp = (const OT*)c.k + page * c.ks[0] + tok * c.ks[1] + hkv * c.ks[2];
    if constexpr (sizeof(OT) == 2) {
        const OT* kr = kp + li * c.ks[1] + 8 * lq;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) t.k[s][kb] = *(const bf16x8*)(kr + 32 * kb);
    } else {
        const OT* kr = kp + li * c.ks[1] + 4 * lq;
#pragma unroll
        for (int kb = 0; kb < D / 16; ++kb) t.k[kb] = *(const f32x4*)(kr + 16 * kb);
    }
}
template <class OT, int D>
__device__ __forceinline__ void attn_load_v(const Cache& c, int u, int hkv, const int (&pg)[2], int s, AttnTile<OT, D>& t) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const int tok = (u * attn_unit<OT>() + 16 * s) & (c.page - 1);
    const long long page = pg[s] >= 0 ? pg[s] : 0;
    const OT* vp = (const OT*)c.v + page * c.vs[0] + tok * c.vs[1] + hkv * c.vs[2];
    if constexpr (sizeof(OT) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t.v[4 * s + i] = *(const typename AttnTile<OT, D>::VT*)(vp + (4 * lq + i) * c.vs[1] + (D / 16) * li);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                t.v[i][j] = *(const f32x4*)(vp + (4 * lq + i) * c.vs[1] + (D / 16) * li + 4 * j);
    }
}
// all of the unit
template <class OT, int D>
__device__ __forceinline__ void attn_load_k(const Cache& c, int u, int hkv, const int (&pg)[2], AttnTile<OT, D>& t) {
#pragma unroll
    for (int s = 0; s < attn_unit<OT>() / 16; ++s) attn_load_k<OT, D>(c, u, hkv, pg, s, t);
}
template <class OT, int D>
__device__ __forceinline__ void attn_load_v(const Cache& c, int u, int hkv, const int (&pg)[2], AttnTile<OT, D>& t) {
#pragma unroll
    for (int s = 0; s < attn_unit<OT>() / 16; ++s) attn_load_v<OT, D>(c, u, hkv, pg, s, t);
}

}  // namespace gdr2
