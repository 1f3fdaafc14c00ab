// Gated delta rule with scalar gates: arguments, workspace layout and sequence maps shared by
// the host launcher and the kernels (internal to libgdr2).
//
//     S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t
//
// with one log-decay g and one write strength beta per token and value head. Inside a chunk of
// 64 tokens with start state S, gam = running sum of g, D_ri = exp(gam_r - gam_i) (i <= r):
//
//     A = strict_lower(beta_r D_ri k_r.k_i)    T = (I + A)^-1    M = lower(D_ri q_r.k_i)
//     X = beta (V - e^gam K S)    Delta = T X    O = e^gam Q S + M Delta
//     S' = e^gamC S + K^T (tail Delta),   tail = exp(gamC - gam)
//
// The decay is one number per row, so it never enters an operand: the raw k, q, v rows (exact in
// the operand type) feed the matrix cores as they are, and every decay factor multiplies an fp32
// accumulator or a row of an intermediate.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdr2_layout.hpp"

namespace gdr2 {

// Per (chunk slot, value head) arrays, id = slot * Hv + head, in the operand type unless said:
//   T     : images (fimg) of T, [NS][64][64]: NS = 2 for bf16, a bf16 value and the bf16 value
//           of what its rounding left over (together 16 bits of mantissa), 1 for fp32
//   M     : image of M, [64][64]
//           (of these triangles' eight fragments of 16 rows and 32 columns, the two that are zero are
//           neither written nor read: sc_img_zero)
//   vec   : fp32 rows of 64: e^gam, beta, tail (all zero in padding rows), gam as a float and its
//           remainder; element 320 is e^gamC
//   training only: T^T and M^T, [NS][64][64] each (the backward chain reads their rows straight into
//   registers; transposed out of LDS instead, they took a quarter of its LDS traffic)
//   training only, each a row of 16-column slices [D / 16][rows][16]:
//   S, dS : chunk start state and end-state gradient, rows = key channels
//   Delta, dY : rows = tokens
struct ScLayout {
    size_t t, m, vec, s, d;                              // element counts per id
    size_t o_t, o_m, o_vec, o_tt, o_mt, o_s, o_ds, o_delta, o_dy;  // byte offsets (T^T, M^T: counts as T)
    size_t o_seg;                                        // segments' ends and transitions, fp32
    size_t infer_bytes, train_bytes;
};

// Fragment (row tile, half of the columns) of a lower (TR: upper) triangular image that is zero.
template <bool TR>
__host__ __device__ constexpr bool sc_img_zero(int rt, int kb) { return TR ? rt >= 2 && kb == 0 : rt < 2 && kb == 1; }

constexpr int SC_E = 0, SC_BETA = 64, SC_TAIL = 128, SC_GHI = 192, SC_GLO = 256, SC_EC = 320, SC_VEC = 384;

constexpr int SC_CHAIN_THREADS = 640;  // of a chain's workgroup: four compute, four side and two producer waves

// segs: segments of all (sequence, value head)s together, 0 where chains are whole
inline ScLayout sc_layout(long long ids, long long segs, int DK, int DV, int esz) {
    ScLayout L;
    const size_t ns = esz == 2 ? 2 : 1;
    L.t = ns * 64 * 64;
    L.m = 64 * 64;
    L.vec = SC_VEC;
    L.s = (size_t)DK * DV;
    L.d = (size_t)64 * DV;
    size_t off = 0;
    auto take = [&](size_t elems, size_t el_bytes) {
        const size_t o = off;
        off += align256((size_t)ids * elems * el_bytes);
        return o;
    };
    L.o_t = take(L.t, esz);
    L.o_m = take(L.m, esz);
    L.o_vec = take(L.vec, 4);
    L.o_seg = off;
    off += align256((size_t)segs * DK * (DV + DK) * sizeof(float));
    L.infer_bytes = off;
    L.o_tt = take(L.t, esz);
    L.o_mt = take(L.t, esz);
    L.o_s = take(L.s, esz);
    L.o_ds = take(L.s, esz);
    L.o_delta = take(L.d, esz);
    L.o_dy = take(L.d, esz);
    L.train_bytes = off;
    return L;
}

struct ScArgs {
    const void *q, *k, *v, *g, *beta;  // [tokens][Hk][DK], [tokens][Hv][DV], [tokens][Hv]
    const float* h0;                   // [N][Hv][DK][DV] or null
    const void* dout;                  // [tokens][Hv][DV]
    const float* dht;                  // [N][Hv][DK][DV] or null
    void* o;                           // null: forward recompute inside the backward
    float* ht;
    void *dq, *dk, *dv, *dg, *dbeta;
    float* dh0;
    const int* cu;                     // packed: [N + 1] on the device, else null
    char* ws;
    ScLayout L;
    int N, T;                          // sequences; tokens of each (packed: tokens in all)
    int Hk, Hv, R;                     // R = Hv / Hk value heads share a key head
    int DK, DV;
    int slots;                         // chunk slots (at least one per chunk of every sequence)
    int nseg, seglen, lead;            // segments of a sequence's chains, their chunks, the first one ahead
    int zero_rest;                     // packed: 1 sets the outputs' rows of no sequence to zero
};

// Segments that chains are cut in, and their chunks: each segment's end from a zero start and its transition
// are found at the same time, joined, and the segments walked together. That is two walks and twice the
// columns (where DK = DV) instead of one, so it pays where walks are few and long: up to 128 of 16 columns,
// with at least 16 chunks a segment, as many segments as give 256 workgroups something, up to 8. lead: the
// first segment is walked in full along with the others' ends, one less to walk after the join, where
// workgroups are short (the ends alone are quicker to find).
// (Packed sequences, whose lengths only the device knows, are walked whole.) Measured, one sequence, bf16,
// d = 128, forward and training step, in segments and whole:
//   16384 tokens  1 head    102 and 295 us,  233 and 645     4 heads   133 and 307,  324 and 679
//                 8 heads   200 and 337,     516 and 771    12 heads   304 and 316,  795 and 910
//    4096 tokens  1 head     57 and 86,      133 and 192     8 heads    79 and 91,   184 and 209
//    2048 tokens  2 heads    52 and 50,      119 and 113 (two segments of 16)
// 8 heads of 16384 tokens without the first segment ahead (four segments): 218 us and 581 us; 1 head with
// it 110 and 241.
inline void sc_segments(int N, int T, int Hv, int DV, bool packed, int& nseg, int& seglen, int& lead) {
    const long long walks = (long long)N * Hv * (DV / 16);
    const int nt = (int)(((long long)T + 63) / 64);
    nseg = 1;
    seglen = nt;
    lead = 0;
    if (packed || walks < 1 || walks > 128) return;
    const int ahead = walks >= 64;
    int n = (int)(256 / walks) + ahead;
    if (n > 8) n = 8;
    if (n > nt / 16) n = nt / 16;
    if (n < 3) return;  // two walks of half the chunks are no shorter
    seglen = (nt + n - 1) / n;
    nseg = (nt + seglen - 1) / seglen;
    lead = ahead;
}

// Sequence s: its first token row, token count and first chunk slot. Packed sequences take the
// slots from start / 64 + s on: as many as they have chunks fit before the next sequence's first.
// cu is data of the caller's that no host check can see, so its entries are held inside the
// tensors here: whatever they are, rows stay below T and slots below `slots`.
struct ScSeq {
    long long tok0;
    int len, nt, slot0;
};
__host__ __device__ __forceinline__ int sc_clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }
__host__ __device__ __forceinline__ ScSeq sc_seq(const int* cu, int T, int s) {
    ScSeq q;
    if (cu) {
        const int b = sc_clamp(cu[s], 0, T), e = sc_clamp(cu[s + 1], b, T);
        q.tok0 = b;
        q.len = e - b;
        q.slot0 = b / 64 + s;
    } else {
        q.tok0 = (long long)s * T;
        q.len = T;
        q.slot0 = s * ((T + 63) / 64);
    }
    q.nt = (q.len + 63) / 64;
    return q;
}
// The sequence whose chunk a slot holds (false: the slot is spare), c its chunk.
__device__ __forceinline__ bool sc_slot(const int* cu, int T, int N, int slot, ScSeq& q, int& c) {
    int s;
    if (cu) {
        int lo = 0, hi = N - 1;  // the last s with slot0(s) <= slot
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sc_clamp(cu[mid], 0, T) / 64 + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
    } else {
        s = slot / ((T + 63) / 64);
    }
    q = sc_seq(cu, T, s);
    c = slot - q.slot0;
    return c >= 0 && c < q.nt;
}

hipError_t launch_sc_fwd(const ScArgs& a, bool bf16, bool train, hipStream_t stream);
hipError_t launch_sc_bwd(const ScArgs& a, bool bf16, hipStream_t stream);
template <class OT, int DK, int DV>
hipError_t launch_sc_fwd_chain_t(const ScArgs& a, bool train, hipStream_t stream);
template <class OT, int DK, int DV>
hipError_t launch_sc_bwd_chain_t(const ScArgs& a, hipStream_t stream);

struct ScStepArgs {
    const void *q, *k, *v, *g, *beta;  // [B][T][Hk][DK], [B][T][Hv][DV], [B][T][Hv]
    float* state;                      // [states][Hv][DK][DV]
    const int* slots;                  // [B] or null: row b's state is slots[b] (null: b)
    void* o;
    int B, T, Hk, Hv, R, states;
    int DK, DV;
    int nt_out;
};
hipError_t launch_sc_step(const ScStepArgs& a, bool bf16, hipStream_t stream);

}  // namespace gdr2
