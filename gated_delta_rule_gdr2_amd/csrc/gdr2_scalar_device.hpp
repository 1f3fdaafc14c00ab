// Device building blocks shared by the kernels of the gated delta rule with scalar gates.
#pragma once
#include "gdr2_device.hpp"
#include "gdr2_scalar.hpp"

namespace gdr2 {

// Operands kept as NS numbers of the operand type: for bf16 a value and what its rounding left
// over, 16 bits of mantissa together (relative error of the pair about 3e-6 in the mean, against
// 1.7e-3 of one bf16), for fp32 the value itself. Intermediates that reach the carried state go
// through the matrix cores this way, so that the state and its gradient, which are fp32, are not
// held to bf16's precision; k, q, v and dO need no second part, being bf16 already.
template <class OT>
struct Split {
    static constexpr int NS = sizeof(OT) == 2 ? 2 : 1;
};
__device__ __forceinline__ void split4(const f32x4& x, bf16x4& hi, bf16x4& lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = (bf16)x[i];
        lo[i] = (bf16)(x[i] - (float)hi[i]);
    }
}

// Exchange fragments in LDS (the contiguous-K order: lane (li, lq) of a 32-deep fragment holds
// K = 8 lq + e of column li as 8 consecutive elements). put_split stores accumulator tile h
// (K rows 16 h .. 16 h + 15) of a fragment as its NS parts, part p at frag + p * stride.
template <class OT>
constexpr int xfrag() { return 64 * 8 * (int)sizeof(OT); }
template <class OT>
__device__ __forceinline__ lds_char* xslot(lds_char* frag, int h) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    return frag + ((li + 16 * (2 * h + (lq >> 1))) * 8 + 4 * (lq & 1)) * (int)sizeof(OT);
}
template <class OT>
__device__ __forceinline__ void put_split(lds_char* frag, int stride, int h, const f32x4& d) {
    lds_char* p = xslot<OT>(frag, h);
    if constexpr (sizeof(OT) == 2) {
        bf16x4 hi, lo;
        split4(d, hi, lo);
        lds_store<bf16x4>(p, hi);
        lds_store<bf16x4>(p + stride, lo);
    } else {
        (void)stride;
        lds_store<f32x4>(p, d);
    }
}
template <class OT>
__device__ __forceinline__ void put_one(lds_char* frag, int h, const f32x4& d) {
    lds_char* p = xslot<OT>(frag, h);
    if constexpr (sizeof(OT) == 2) {
        bf16x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (bf16)d[i];
        lds_store<bf16x4>(p, x);
    } else {
        lds_store<f32x4>(p, d);
    }
}
template <class OT>
__device__ __forceinline__ typename Frag<OT>::type get_x(const lds_char* frag) {
    return lds_load<typename Frag<OT>::type>(frag + lane_id() * 8 * (int)sizeof(OT));
}

// Rows 16 kt .. + 15 (K rows, kt = 0 or 1) of an exchange fragment's first part (bf16), turned for a
// 16-column slice [rows][16]: a transposing read gives lane (li, lq) columns 4 lq .. + 3 of row 16 kt + li.
__device__ __forceinline__ bf16x4 read_slice_tr(const lds_char* frag, int kt) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const int r = 4 * lq + (li >> 2), c = 16 * kt + 4 * (li & 3);  // column r, K index c .. c + 3
    return lds_read_tr16(frag + ((r + 16 * (c >> 3)) * 8 + (c & 7)) * 2);
}

// This lane's row and K group, as values the compiler cannot trace back to the thread index. The
// kernels below run long phases, each with its own set of swizzled LDS addresses; left to itself
// the compiler computes all of them once, ahead of the loop over value heads, keeps them in some
// hundred registers and spills. Each phase starts from its own copy instead.
struct Lane {
    int li, lq;
};
__device__ __forceinline__ Lane fresh_lane() {
    int l = lane_id();
    asm volatile("" : "+v"(l));
    return {l & 15, l >> 4};
}
// fragment reads as lfrag_rowk8 / lfrag_colk8 (gdr2_device.hpp), for a given Lane
template <class OT, class V>
__device__ __forceinline__ typename Frag<OT>::type frag_rows(const Lane& n, const V& m, int row0, int k0) {
    const lds_char* p0 = m.p + m.off(row0 + n.li, k0 + 8 * n.lq);
    if constexpr (sizeof(OT) == 2) {
        return lds_load<bf16x8>(p0);
    } else {
        const f32x4 x0 = lds_load<f32x4>(p0), x1 = lds_load<f32x4>(m.p + m.off(row0 + n.li, k0 + 8 * n.lq + 4));
        return __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}
template <class OT, class V>
__device__ __forceinline__ typename Frag<OT>::type frag_cols(const Lane& n, const V& m, int col0, int k0) {
    if constexpr (sizeof(OT) == 2) {
        const int r = k0 + 8 * n.lq + (n.li >> 2), c = col0 + 4 * (n.li & 3);
        const bf16x4 v0 = lds_read_tr16(m.p + m.off(r, c)), v1 = lds_read_tr16(m.p + m.off(r + 4, c));
        return __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        typename Frag<OT>::type f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = lds_load<float>(m.p + m.off(k0 + 8 * n.lq + e, col0 + n.li));
        return f;
    }
}

// Sum over the four lanes li + 16 lq of a column, in all of them: two exchanges of half waves and of
// neighbouring rows in the vector unit, without the LDS round trip of a shuffle.
__device__ __forceinline__ float sum_lq(float x) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// value of lane n (a constant) in every lane
__device__ __forceinline__ float lane_value(float x, int n) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), n));
}

// Fragments of a slice array [D / 16][rows][16] (row-K, the contiguous K order): row row0 + li,
// columns 32 kb + 8 lq .. + 7.
template <class OT, int ROWS>
__device__ __forceinline__ int slice_off(int row, int c) { return ((c >> 4) * ROWS + row) * 16 + (c & 15); }
template <class OT, int ROWS>
__device__ __forceinline__ typename Frag<OT>::type gfrag_slice(const OT* m, int row0, int kb) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const OT* p = m + slice_off<OT, ROWS>(row0 + li, 32 * kb + 8 * lq);
    if constexpr (sizeof(OT) == 2) {
        return *(const bf16x8*)p;
    } else {
        const f32x4 x0 = *(const f32x4*)p, x1 = *(const f32x4*)(p + 4);
        return __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}
template <class OT, int ROWS>
struct LSlice {  // the same array in LDS
    const lds_char* p;
    __device__ __forceinline__ int off(int r, int c) const { return slice_off<OT, ROWS>(r, c) * (int)sizeof(OT); }
};

// Packed, zero_rest: the rows of [.][heads][D] outputs that lie before the first or behind the last
// sequence, of the 64 rows from 64 slot on, heads h0 .. h0 + nh - 1, set to zero (workgroup slot of
// the grid; the slots are at least as many as the 64-row pieces of the tensors).
template <class OT>
__device__ __forceinline__ void zero_rest_rows(const ScArgs& a, int slot, void* p, int heads, int h0, int nh, int D) {
    const int b = sc_clamp(a.cu[0], 0, a.T), e = sc_clamp(a.cu[a.N], b, a.T);
    const int r0 = 64 * slot, r1 = min(r0 + 64, a.T);
    if (r0 >= b && r1 <= e) return;
    for (int i = threadIdx.x; i < 64 * nh * D; i += blockDim.x) {
        const int r = r0 + i / (nh * D), x = i % (nh * D);
        if (r < r1 && (r < b || r >= e)) ((OT*)p)[((size_t)r * heads + h0) * D + x] = to_ot<OT>(0.f);
    }
}

}  // namespace gdr2
