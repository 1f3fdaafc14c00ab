// Device building blocks of attention over whole sequences: 32x32 matrix products and the tiles they read.
//
// Products are built from 32x32 output tiles with 16-deep K blocks: one v_mfma_f32_32x32x16_bf16, or eight
// v_mfma_f32_32x32x2_f32. Lane l = li + 32 h (li = l % 32, h = l / 32) holds 8 elements of an operand: row (A) or
// column (B) li, and K indices 8 h + e in the contiguous order, or 8 (e / 4) + 4 h + e % 4 in the accumulator's. An
// accumulator holds rows 8 (r / 4) + 4 h + r % 4, r = 0 .. 15, of column li; so registers 8 b .. 8 b + 7 are, in the
// accumulator's order, the B operand of the K block 16 b .. 16 b + 15: scores become weights and enter the next
// product where they stand.
//
// A 32x32 product takes 32 clocks for two operands of 16 bytes a lane, a 16x16x32 one 16 clocks: half the LDS
// traffic, which with 16x16 tiles would be what bounds these kernels.
#pragma once
#include "gdr2_device.hpp"
#include "gdr2_prompt.hpp"

namespace gdr2 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void mma32(f32x16& acc, const bf16x8& a, const bf16x8& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma32(f32x16& acc, const f32x8& a, const f32x8& b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    return x;
}

// Tiles in LDS: rows of D elements, their 16-byte chunks permuted by an XOR with tile_f(row). A 16-byte read is served
// in passes of 16 lanes, an 8-byte one of 32 (gdr2_device.hpp); the row reads of a 32x32 operand (row li, chunk
// c + h) have in a pass the rows whose bits 4..2 have even (odd) parity, and the transposing reads four rows and four
// chunks. Both cover distinct banks with
//   16 chunks a row: f(r) = 4 (r mod 4) + (r / 4 mod 4)     8 chunks: f(r) = 4 (r / 2 mod 2) + (r / 4 mod 4)
// (fp32, 32 chunks: as 16; its transposing reads are single floats and two lanes share a bank).
template <int NCH>
__device__ __forceinline__ int tile_f(int r) {
    static_assert(NCH == 8 || NCH == 16 || NCH == 32, "tiles have 8, 16 or 32 chunks a row");
    return NCH == 8 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : 4 * (r & 3) + ((r >> 2) & 3);
}
template <class OT, int D>
struct Tile32 {
    static constexpr int ES = (int)sizeof(OT), EPC = 16 / ES, NCH = D / EPC, RB = D * ES;  // row bytes
    static __device__ __forceinline__ int off(int r, int c) {
        return r * RB + (((c / EPC) ^ tile_f<NCH>(r)) * 16) + (c % EPC) * ES;
    }
    // A operand of the K block k0 .. k0 + 15, rows r0 + li, contiguous K order
    static __device__ __forceinline__ typename Frag<OT>::type rows(const lds_char* t, int r0, int k0) {
        const int l = lane_id(), r = r0 + (l & 31), c = k0 + 8 * (l >> 5);
        if constexpr (ES == 2) {
            return lds_load<bf16x8>(t + off(r, c));
        } else {
            const f32x4 x0 = lds_load<f32x4>(t + off(r, c)), x1 = lds_load<f32x4>(t + off(r, c + 4));
            return __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // A operand of the transposed tile: rows are the tile's columns c0 + li, the K block its rows k0 .. k0 + 15 in
    // the accumulator's order
    static __device__ __forceinline__ typename Frag<OT>::type cols(const lds_char* t, int c0, int k0) {
        const int l = lane_id(), h = l >> 5;
        if constexpr (ES == 2) {
            const int r = k0 + 4 * h + ((l & 15) >> 2), c = c0 + 16 * ((l >> 4) & 1) + 4 * (l & 3);
            const bf16x4 v0 = lds_read_tr16(t + off(r, c)), v1 = lds_read_tr16(t + off(r + 8, c));
            return __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            typename Frag<OT>::type f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = lds_load<float>(t + off(k0 + 8 * (e >> 2) + 4 * h + (e & 3), c0 + (l & 31)));
            return f;
        }
    }
    // Rows row0 .. row0 + R - 1 (held in 0 .. last) of a matrix with row stride rs (bytes) into LDS, 1 KB a wave
    // instruction, wave w of NW
    template <int R, int NW>
    static __device__ __forceinline__ void load(const char* base, long long rs, int row0, int last, lds_char* t, int w) {
        constexpr int N = R * RB / 1024, RPI = 64 / NCH > 0 ? 64 / NCH : 1;
        const int l = lane_id();
        static_assert(NCH <= 64 && R * RB % 1024 == 0, "whole rows an instruction");
#pragma unroll
        for (int i = 0; i < (N + NW - 1) / NW; ++i) {
            const int n = i * NW + w;
            if (N % NW == 0 || n < N) {
                const int r = n * RPI + l / NCH;
                const int row = max(0, min(row0 + r, last));
                const char* src = base + (long long)row * rs + (((l % NCH) ^ tile_f<NCH>(r)) * 16);
                __builtin_amdgcn_global_load_lds(src, (lds_void*)(t + n * 1024), 16, 0, 0);
            }
        }
    }
};

// B operands of a wave's own 32 rows, all K blocks, straight from memory: row p (this lane's), contiguous K order.
template <class OT, int D>
__device__ __forceinline__ void load_own(const OT* p, bool neg, typename Frag<OT>::type (&f)[D / 16]) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int kb = 0; kb < D / 16; ++kb) {
        f[kb] = *(const typename Frag<OT>::type*)(p + 16 * kb + 8 * h);
        if (neg) f[kb] = -f[kb];
    }
}
// registers 8 b .. 8 b + 7 of an accumulator as the B operand of K block b
template <class OT>
__device__ __forceinline__ typename Frag<OT>::type acc_frag(const f32x16& x, int b) {
    typename Frag<OT>::type f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_ot<OT>(x[8 * b + e]);
    return f;
}
// this lane's column of D rows, held in accumulators, times f: four consecutive elements at a time
template <class OT, int D>
__device__ __forceinline__ void store_col(OT* p, const f32x16 (&acc)[D / 32], float f) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x[4] = {acc[dt][4 * j] * f, acc[dt][4 * j + 1] * f, acc[dt][4 * j + 2] * f, acc[dt][4 * j + 3] * f};
            st4(p + 32 * dt + 8 * j + 4 * h, x);
        }
}
// the other half wave's value of this column
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// The sequence tile a workgroup works on.
struct PromptAt {
    long long tok0;  // the sequence's first token
    int len, tile;   // its tokens; which of its tiles
    bool any;        // false: a spare slot
};
__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
// Packed: the sequence whose tile a slot holds. cu is data of the caller's that no host check can see, so its entries
// are held inside the tensors here.
__device__ __forceinline__ PromptAt prompt_packed(const PromptArgs& a, int slot, int tile) {
    int lo = 0, hi = a.N - 1;  // the last sequence whose first slot is not behind it
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (clamp_int(a.cu[mid], 0, a.T) / tile + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    const int b = clamp_int(a.cu[lo], 0, a.T), e = clamp_int(a.cu[lo + 1], b, a.T);
    PromptAt p;
    p.tok0 = b;
    p.len = e - b;
    p.tile = slot - (b / tile + lo);
    p.any = p.tile >= 0 && (long long)p.tile * tile < p.len;
    return p;
}
// Tiles in the order of the launch: the last tile of every sequence first (`last_first`), which sees the most keys, or
// the first one first, which is seen most. `heads` workgroups a tile; heads that share keys lie a multiple of the
// key heads apart, mostly on one XCD. Returns the head's place 0 .. heads - 1, key heads innermost.
__device__ __forceinline__ int prompt_at(const PromptArgs& a, int bid, int tile, int heads, bool last_first, PromptAt& p,
                                         int& slot) {
    if (a.cu) {
        const int ns = a.T / tile + a.N, s = bid / heads;
        slot = last_first ? ns - 1 - s : s;
        p = prompt_packed(a, slot, tile);
        return bid % heads;
    }
    const int nt = (a.T + tile - 1) / tile, cols = a.N * heads, t = bid / cols, c = bid % cols;
    // c: group of heads outermost, then sequences, then key heads
    const int per = a.N * a.Hkv, g = c / per, s = c % per / a.Hkv, hk = c % a.Hkv;
    p.tile = last_first ? nt - 1 - t : t;
    p.tok0 = (long long)s * a.T;
    p.len = a.T;
    p.any = true;
    slot = 0;
    return g * a.Hkv + hk;
}
// Packed, zero_rest: rows of no sequence among rows tile * slot .. of a [tokens][heads][D] output, one head, set to zero.
template <class OT>
__device__ __forceinline__ void prompt_zero(const PromptArgs& a, int slot, int tile, OT* p, int heads, int head, int D) {
    const int b = clamp_int(a.cu[0], 0, a.T), e = clamp_int(a.cu[a.N], b, a.T);
    const int r0 = min((long long)tile * slot, (long long)a.T), r1 = min(r0 + tile, a.T);
    if (r0 >= b && r1 <= e) return;
    for (int i = threadIdx.x; i < (r1 - r0) * D; i += blockDim.x) {
        const int r = r0 + i / D;
        if (r < b || r >= e) p[((long long)r * heads + head) * D + i % D] = to_ot<OT>(0.f);
    }
}

}  // namespace gdr2
