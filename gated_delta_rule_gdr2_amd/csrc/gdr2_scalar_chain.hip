// Gated delta rule with scalar gates: the two sequential chains (equations in gdr2_scalar.hpp).
//
//   forward  : Y = K S ;  X = beta (V - e^gam Y) ;  Delta = T X ;
//              O = e^gam Q S + M Delta ;  S' = e^gamC S + K^T (tail Delta)
//   backward : dDelta = M^T dO + tail K dS' ;  dY = T^T dDelta ;
//              dS = e^gamC dS' + Q^T (e^gam dO) - K^T (beta e^gam dY)
//
// Each (sequence, value head, 16 value columns) is its own chain over the chunks: one workgroup of
// four compute waves and two producer waves. Compute wave w owns token tile w and d_k / 4 key rows
// of the state slice, which stay in fp32 accumulators for the whole walk. A step is three products
// that follow one another, with the intermediate published through LDS between them (three
// barriers): the state slice, X (dDelta), and Delta (beta e^gam dY). Everything that reaches the
// state goes through as NS parts (Split in gdr2_scalar_device.hpp): the state and its gradient come
// out to about 5e-6, at two to four bf16 products for one, on matrix cores that wait for operands
// most of the time anyway.
//
// Against the chains of the channel-wise operator, which read five per-chunk matrices that their
// intra-chunk kernel wrote (W_m, K_d^T, Q_g, M, U), these read the caller's own q, k, v and T, M:
// the scalar decay scales accumulators instead of operands, so K S and K^T Delta share one raw K tile
// in LDS (read by rows and, transposed, by columns), and value heads that share a key head share
// its rows in L2.
//
// The producers stream a chunk's operands into LDS by asynchronous DMA, 16 bytes a lane, into two
// buffers, the next chunk's while this one's step runs.
#include "gdr2_intra_common.hpp"
#include "gdr2_scalar_device.hpp"

namespace gdr2 {

constexpr int SC_NC = 4;  // compute waves
constexpr int SC_NP = 2;  // producer waves

__device__ __forceinline__ int sc_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Producer pi's share of a copy of BYTES (a multiple of 1024) into LDS: 1 KB pieces pi, pi + SC_NP, ...
template <int BYTES>
__device__ __forceinline__ void sc_dma(const void* src, lds_char* dst, int pi) {
    static_assert(BYTES % 1024 == 0, "whole kilobytes");
    const int l = lane_id();
#pragma unroll
    for (int k = 0; k < BYTES / 1024; ++k)
        if (k % SC_NP == pi)
            __builtin_amdgcn_global_load_lds((const char*)src + k * 1024 + l * 16, (lds_void*)(dst + k * 1024), 16, 0, 0);
}
// ... of the 64 rows of a row-major tensor (row stride rs elements, RL read of each) into a
// swizzled tile. Rows from nvalid on repeat the last valid one: every product multiplies them by
// rows of beta, tail, e^gam, M or Delta that are exact zeros, and a caller's padding is not read.
template <class OT, int RL>
__device__ __forceinline__ void sc_dma_rows(const OT* base, size_t rs, int nvalid, lds_char* tile, int pi) {
    constexpr int EPC = 16 / (int)sizeof(OT), NCH = RL / EPC, RPI = 64 / NCH;
    const int l = lane_id();
#pragma unroll
    for (int n = 0; n < CH / RPI; ++n) {
        if (n % SC_NP == pi) {
            const int row = n * RPI + l / NCH, c = (l % NCH) ^ swz_f<OT, RL>(row);
            const char* src = (const char*)(base + (size_t)min(row, nvalid - 1) * rs + c * EPC);
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(tile + n * 1024), 16, 0, 0);
        }
    }
}
// ... of a 16-column slice of the 64 rows, as [64][16]
template <class OT>
__device__ __forceinline__ void sc_dma_slice(const OT* base, size_t rs, int nvalid, lds_char* tile, int pi) {
    constexpr int EPC = 16 / (int)sizeof(OT), LPR = 16 / EPC, RPI = 64 / LPR;
    const int l = lane_id();
#pragma unroll
    for (int n = 0; n < CH / RPI; ++n) {
        if (n % SC_NP == pi) {
            const int row = n * RPI + l / LPR;
            const char* src = (const char*)(base + (size_t)min(row, nvalid - 1) * rs + (l % LPR) * EPC);
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(tile + n * 1024), 16, 0, 0);
        }
    }
}

// chain workgroup -> (sequence, value head, slice): workgroups go to the 8 XCDs round-robin, so
// that the slices of a (sequence, head), which read the same q, k, T and M, share an L2, as far as
// their number allows
__device__ __forceinline__ void sc_chain_map(int gid, int pairs, int NJ, int& s, int& j) {
    if (pairs % 8 == 0) {
        const int x = gid % 8, rest = gid / 8;
        j = rest % NJ;
        s = (rest / NJ) * 8 + x;
    } else {
        s = gid / NJ;
        j = gid % NJ;
    }
}

template <class OT, int DK, bool BWD>
struct ScChainLds {  // one operand buffer, and the exchange
    static constexpr int ES = sizeof(OT), NS = Split<OT>::NS, NKB = DK / 32;
    static constexpr int SQ = CH * CH * ES;
    static constexpr int K = 0;
    static constexpr int Q = K + CH * DK * ES;
    static constexpr int V = Q + CH * DK * ES;        // v (forward) or dO (backward), [64][16]
    static constexpr int T = V + CH * 16 * ES;        // NS images
    static constexpr int M = T + NS * SQ;             // 1 image (forward), NS (backward)
    static constexpr int VEC = M + (BWD ? NS : 1) * SQ;
    static constexpr int BYTES = VEC + 2048;          // SC_VEC floats, in whole kilobytes
    static constexpr int F = xfrag<OT>();
    static constexpr int XS = 0;                      // state slice: NS x NKB fragments
    static constexpr int XX = XS + NS * NKB * F;      // X or dDelta: NS x 2
    static constexpr int XD = XX + NS * 2 * F;        // tail Delta or beta e^gam dY: NS x 2
    static constexpr int XO = XD + NS * 2 * F;        // Delta or dY, one part: 2
    static constexpr int XBYTES = XO + 2 * F;
    static_assert(2 * BYTES + XBYTES <= 160 * 1024, "two operand buffers fit");
};

// Where a walk finds its data.
template <class OT>
struct ScWalk {
    ScSeq q;
    int h, hk, j;
    const float* start;
    float* end;
};

// A producer's side: the operands of chunk index(n), n = 0 .. nt - 1, into buffer n % 2. Takes part
// in the step's barriers.
template <class OT, int DK, int DV, bool BWD>
__device__ __forceinline__ void sc_produce(const ScArgs& a, const ScWalk<OT>& w, lds_char* b0, lds_char* b1, int pi) {
    using B = ScChainLds<OT, DK, BWD>;
    const int nt = w.q.nt;
    const size_t rsk = (size_t)a.Hk * DK, rsv = (size_t)a.Hv * DV;
    auto load = [&](int n) {
        const int c = BWD ? nt - 1 - n : n;
        lds_char* buf = (n & 1) ? b1 : b0;
        const long long row0 = w.q.tok0 + 64LL * c;
        const int nvalid = min(CH, w.q.len - CH * c);
        const size_t id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        sc_dma_rows<OT, DK>((const OT*)a.k + row0 * rsk + (size_t)w.hk * DK, rsk, nvalid, buf + B::K, pi);
        const OT* v = BWD ? (const OT*)a.dout : (const OT*)a.v;
        sc_dma_slice<OT>(v + row0 * rsv + (size_t)w.h * DV + 16 * w.j, rsv, nvalid, buf + B::V, pi);
        if (pi == 1) {  // the row factors: 1.5 KB of the 2 KB the buffer has for them
            const char* src = a.ws + a.L.o_vec + id * a.L.vec * 4;
            __builtin_amdgcn_global_load_lds(src + lane_id() * 16, (lds_void*)(buf + B::VEC), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(src + 1024 + (lane_id() & 31) * 16, (lds_void*)(buf + B::VEC + 1024), 16, 0,
                                             0);
        }
        sc_dma<B::NS * B::SQ>(a.ws + a.L.o_t + id * a.L.t * B::ES, buf + B::T, pi);
        if (BWD || a.o) {
            sc_dma_rows<OT, DK>((const OT*)a.q + row0 * rsk + (size_t)w.hk * DK, rsk, nvalid, buf + B::Q, pi);
            sc_dma<(BWD ? B::NS : 1) * B::SQ>(a.ws + a.L.o_m + id * a.L.m * B::ES, buf + B::M, pi);
        }
    };
    load(0);
    wait_vm<0>();
    for (int n = 0; n < nt; ++n) {
        sync_lds();  // A: chunk n is in its buffer; the other buffer (chunk n - 1) is free
        if (n + 1 < nt) load(n + 1);
        sync_lds();  // B
        sync_lds();  // C
        wait_vm<0>();
    }
}

template <class OT, int DK, int DV, bool TRAIN, bool OUT>
__device__ __forceinline__ void sc_fwd_walk(const ScArgs& a, const ScWalk<OT>& w, lds_char* b0, lds_char* b1,
                                            lds_char* xs) {
    using B = ScChainLds<OT, DK, false>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F, NT = DK / 64;  // NT: 16-row state tiles of a wave
    const int wv = sc_wave(), l = lane_id(), li = l & 15, lq = l >> 4;
    const int nt = w.q.nt;
    // state tile t: key rows 16 (NT wv + t) + 4 lq + i, column 16 j + li
    f32x4 S[NT];
    auto publish_state = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int rt = NT * wv + t;
            put_split<OT>(xs + B::XS + (rt >> 1) * F, NKB * F, rt & 1, S[t]);
        }
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            S[t][i] = w.start ? w.start[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * DV + 16 * w.j + li] : 0.f;
    publish_state();
#pragma unroll 1
    for (int n = 0; n < nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vK{buf + B::K}, vQ{buf + B::Q};
        const LImg<OT, CH> vM{buf + B::M};
        const size_t id = (size_t)(w.q.slot0 + n) * a.Hv + w.h;
        sync_lds();  // A: the state slice is published, the chunk's operands are in
        FT SB[NS][NKB];
#pragma unroll
        for (int p = 0; p < NS; ++p)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) SB[p][kb] = get_x<OT>(xs + B::XS + (p * NKB + kb) * F);
        float e4[4], b4[4], t4[4];
        lds_get4<float>(buf + B::VEC + (SC_E + 16 * wv + 4 * lq) * 4, e4);
        lds_get4<float>(buf + B::VEC + (SC_BETA + 16 * wv + 4 * lq) * 4, b4);
        lds_get4<float>(buf + B::VEC + (SC_TAIL + 16 * wv + 4 * lq) * 4, t4);
        // X = beta (V - e^gam K S) on this wave's tokens
        f32x4 Y = {0.f, 0.f, 0.f, 0.f}, Y1 = Y;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            const FT k = lfrag_rowk8<OT>(vK, 16 * wv, 32 * kb);
            mma(Y, k, SB[0][kb]);
            if constexpr (NS == 2) mma(Y1, k, SB[1][kb]);
        }
        f32x4 X;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = lds_get1<OT>(buf + B::V + ((16 * wv + 4 * lq + i) * 16 + li) * B::ES);
            X[i] = b4[i] * (v - e4[i] * (Y[i] + Y1[i]));
        }
        put_split<OT>(xs + B::XX + (wv >> 1) * F, 2 * F, wv & 1, X);
        // the state's part of O^T (rows: value columns, columns: tokens)
        f32x4 O = {0.f, 0.f, 0.f, 0.f};
        if (OUT) {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) mma(O, SB[0][kb], lfrag_rowk8<OT>(vQ, 16 * wv, 32 * kb));
            O = O * lds_load<float>(buf + B::VEC + (SC_E + 16 * wv + li) * 4);
        }
        if (TRAIN) {  // the chunk's start state, this wave's key rows
            OT* s = (OT*)(a.ws + a.L.o_s) + id * a.L.s + (size_t)w.j * DK * 16;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int rt = NT * wv + t;
                if constexpr (NS == 2) store_slice_tr(xs + B::XS + (rt >> 1) * F, rt & 1, s + rt * 256);
                else store_slice_acc<OT>(S[t], s + rt * 256);
            }
        }
        sync_lds();  // B: X is published
        // Delta = T X on this wave's tokens (T is lower triangular: token tiles 0 and 1 need only
        // the first 32 columns)
        f32x4 D = {0.f, 0.f, 0.f, 0.f}, D1 = D;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb == 0 || wv >= 2) {
#pragma unroll
                for (int p = 0; p < NS; ++p) {
                    const FT t = lfrag_rowk8<OT>(LImg<OT, CH>{buf + B::T + p * B::SQ}, 16 * wv, 32 * kb);
                    mma(D, t, get_x<OT>(xs + B::XX + kb * F));
                    if constexpr (NS == 2) mma(D1, t, get_x<OT>(xs + B::XX + (2 + kb) * F));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            D[i] += D1[i];
            D1[i] = t4[i] * D[i];
        }
        put_split<OT>(xs + B::XD + (wv >> 1) * F, 2 * F, wv & 1, D1);
        if (OUT || TRAIN) put_one<OT>(xs + B::XO + (wv >> 1) * F, wv & 1, D);
        const float ec = lds_load<float>(buf + B::VEC + SC_EC * 4);
        sync_lds();  // C: Delta is published
        FT DB[NS][2];
#pragma unroll
        for (int p = 0; p < NS; ++p)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) DB[p][kb] = get_x<OT>(xs + B::XD + (2 * p + kb) * F);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 s0 = S[t] * ec, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const FT k = lfrag_colk8<OT>(vK, 16 * (NT * wv + t), 32 * kb);
                mma(s0, k, DB[0][kb]);
                if constexpr (NS == 2) mma(s1, k, DB[1][kb]);
            }
            S[t] = s0 + s1;
        }
        publish_state();
        if (OUT) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 0 || wv >= 2)
                    mma(O, get_x<OT>(xs + B::XO + kb * F), lfrag_rowk8<OT>(vM, 16 * wv, 32 * kb));
            const int row = 16 * wv + li;
            if (CH * n + row < w.q.len) {
                const float ov[4] = {O[0], O[1], O[2], O[3]};
                st4((OT*)a.o + ((size_t)(w.q.tok0 + 64LL * n + row) * a.Hv + w.h) * DV + 16 * w.j + 4 * lq, ov);
            }
        }
        if (TRAIN) {
            OT* d = (OT*)(a.ws + a.L.o_delta) + id * a.L.d + (size_t)w.j * CH * 16 + wv * 256;
            if constexpr (NS == 2) store_slice_tr(xs + B::XO + (wv >> 1) * F, wv & 1, d);
            else store_slice_acc<OT>(D, d);
        }
    }
    if (w.end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w.end[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * DV + 16 * w.j + li] = S[t][i];
    }
}

template <class OT, int DK, int DV>
__device__ __forceinline__ void sc_walk_of(const ScArgs& a, ScWalk<OT>& w, size_t& st) {
    int p;
    sc_chain_map(blockIdx.x, a.N * a.Hv, DV / 16, p, w.j);
    const int s = p / a.Hv;
    w.h = p % a.Hv;
    w.hk = w.h / a.R;
    w.q = sc_seq(a.cu, a.T, s);
    st = (size_t)p * DK * DV;
}

template <class OT, int DK, int DV, bool TRAIN, bool OUT>
__global__ __launch_bounds__(64 * (SC_NC + SC_NP)) void k_sc_fwd_chain(ScArgs a) {
    using B = ScChainLds<OT, DK, false>;
    __shared__ __align__(16) char buf0[B::BYTES];
    __shared__ __align__(16) char buf1[B::BYTES];
    __shared__ __align__(16) char xch[B::XBYTES];
    poison_lds((lds_char*)buf0, sizeof(buf0));
    poison_lds((lds_char*)buf1, sizeof(buf1));
    poison_lds((lds_char*)xch, sizeof(xch));
    poison_lds_done();
    ScWalk<OT> w;
    size_t st;
    sc_walk_of<OT, DK, DV>(a, w, st);
    w.start = a.h0 ? a.h0 + st : nullptr;
    w.end = a.ht ? a.ht + st : nullptr;
    const int wv = sc_wave();
    if (wv >= SC_NC) {
        if (w.q.nt > 0) sc_produce<OT, DK, DV, false>(a, w, (lds_char*)buf0, (lds_char*)buf1, wv - SC_NC);
        return;
    }
    sc_fwd_walk<OT, DK, DV, TRAIN, OUT>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
}

template <class OT, int DK, int DV>
__device__ __forceinline__ void sc_bwd_walk(const ScArgs& a, const ScWalk<OT>& w, lds_char* b0, lds_char* b1,
                                            lds_char* xs) {
    using B = ScChainLds<OT, DK, true>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F, NT = DK / 64;
    const int wv = sc_wave(), l = lane_id(), li = l & 15, lq = l >> 4;
    const int nt = w.q.nt;
    f32x4 dS[NT];
    auto publish_state = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int rt = NT * wv + t;
            put_split<OT>(xs + B::XS + (rt >> 1) * F, NKB * F, rt & 1, dS[t]);
        }
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dS[t][i] = w.start ? w.start[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * DV + 16 * w.j + li] : 0.f;
    publish_state();
#pragma unroll 1
    for (int n = 0; n < nt; ++n) {
        const int c = nt - 1 - n;
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vK{buf + B::K}, vQ{buf + B::Q};
        const LPad<OT> vO{buf + B::V, 16};
        const size_t id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        sync_lds();  // A: the end-state gradient is published, the chunk's operands are in
        float e4[4], b4[4], t4[4];
        lds_get4<float>(buf + B::VEC + (SC_E + 16 * wv + 4 * lq) * 4, e4);
        lds_get4<float>(buf + B::VEC + (SC_BETA + 16 * wv + 4 * lq) * 4, b4);
        lds_get4<float>(buf + B::VEC + (SC_TAIL + 16 * wv + 4 * lq) * 4, t4);
        // dDelta = tail K dS' + M^T dO on this wave's tokens (M^T is upper triangular: token tiles 2
        // and 3 need only the last 32 rows)
        f32x4 Y = {0.f, 0.f, 0.f, 0.f}, Y1 = Y;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            const FT k = lfrag_rowk8<OT>(vK, 16 * wv, 32 * kb);
            mma(Y, k, get_x<OT>(xs + B::XS + kb * F));
            if constexpr (NS == 2) mma(Y1, k, get_x<OT>(xs + B::XS + (NKB + kb) * F));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[i] = t4[i] * (Y[i] + Y1[i]);
        FT dO[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) dO[kb] = lfrag_colk8<OT>(vO, 0, 32 * kb);
        Y1 = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb == 1 || wv < 2) {
                mma(Y, lfrag_colk8<OT>(LImg<OT, CH>{buf + B::M}, 16 * wv, 32 * kb), dO[kb]);
                if constexpr (NS == 2)
                    mma(Y1, lfrag_colk8<OT>(LImg<OT, CH>{buf + B::M + B::SQ}, 16 * wv, 32 * kb), dO[kb]);
            }
        }
        put_split<OT>(xs + B::XX + (wv >> 1) * F, 2 * F, wv & 1, Y + Y1);
        {  // the chunk's end-state gradient, this wave's key rows
            OT* s = (OT*)(a.ws + a.L.o_ds) + id * a.L.s + (size_t)w.j * DK * 16;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int rt = NT * wv + t;
                if constexpr (NS == 2) store_slice_tr(xs + B::XS + (rt >> 1) * F, rt & 1, s + rt * 256);
                else store_slice_acc<OT>(dS[t], s + rt * 256);
            }
        }
        // the part of dS without dY: e^gamC dS' + Q^T (e^gam dO)
        const float ec = lds_load<float>(buf + B::VEC + SC_EC * 4);
        f32x4 P[NT], P1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            P[t] = dS[t] * ec;
            P1[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            FT hi, lo;
            float s8[8];
            lds_get4<float>(buf + B::VEC + (SC_E + 32 * kb + 8 * lq) * 4, s8);
            lds_get4<float>(buf + B::VEC + (SC_E + 32 * kb + 8 * lq + 4) * 4, s8 + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = s8[e] * to_f(dO[kb][e]);
                hi[e] = to_ot<OT>(x);
                lo[e] = to_ot<OT>(x - to_f(hi[e]));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const FT qt = lfrag_colk8<OT>(vQ, 16 * (NT * wv + t), 32 * kb);
                mma(P[t], qt, hi);
                if constexpr (NS == 2) mma(P1[t], qt, lo);
            }
        }
        sync_lds();  // B: dDelta is published
        f32x4 D = {0.f, 0.f, 0.f, 0.f}, D1 = D;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (kb == 1 || wv < 2) {
#pragma unroll
                for (int p = 0; p < NS; ++p) {
                    const FT t = lfrag_colk8<OT>(LImg<OT, CH>{buf + B::T + p * B::SQ}, 16 * wv, 32 * kb);
                    mma(D, t, get_x<OT>(xs + B::XX + kb * F));
                    if constexpr (NS == 2) mma(D1, t, get_x<OT>(xs + B::XX + (2 + kb) * F));
                }
            }
        }
        f32x4 Z;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            D[i] += D1[i];
            Z[i] = -(b4[i] * e4[i]) * D[i];
        }
        put_split<OT>(xs + B::XD + (wv >> 1) * F, 2 * F, wv & 1, Z);
        put_one<OT>(xs + B::XO + (wv >> 1) * F, wv & 1, D);
        sync_lds();  // C: dY is published
        FT DB[NS][2];
#pragma unroll
        for (int p = 0; p < NS; ++p)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) DB[p][kb] = get_x<OT>(xs + B::XD + (2 * p + kb) * F);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const FT k = lfrag_colk8<OT>(vK, 16 * (NT * wv + t), 32 * kb);
                mma(P[t], k, DB[0][kb]);
                if constexpr (NS == 2) mma(P1[t], k, DB[1][kb]);
            }
            dS[t] = P[t] + P1[t];
        }
        publish_state();
        OT* d = (OT*)(a.ws + a.L.o_dy) + id * a.L.d + (size_t)w.j * CH * 16 + wv * 256;
        if constexpr (NS == 2) store_slice_tr(xs + B::XO + (wv >> 1) * F, wv & 1, d);
        else store_slice_acc<OT>(D, d);
    }
    if (w.end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w.end[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * DV + 16 * w.j + li] = dS[t][i];
    }
}

template <class OT, int DK, int DV>
__global__ __launch_bounds__(64 * (SC_NC + SC_NP)) void k_sc_bwd_chain(ScArgs a) {
    using B = ScChainLds<OT, DK, true>;
    __shared__ __align__(16) char buf0[B::BYTES];
    __shared__ __align__(16) char buf1[B::BYTES];
    __shared__ __align__(16) char xch[B::XBYTES];
    poison_lds((lds_char*)buf0, sizeof(buf0));
    poison_lds((lds_char*)buf1, sizeof(buf1));
    poison_lds((lds_char*)xch, sizeof(xch));
    poison_lds_done();
    ScWalk<OT> w;
    size_t st;
    sc_walk_of<OT, DK, DV>(a, w, st);
    w.start = a.dht ? a.dht + st : nullptr;
    w.end = a.dh0 ? a.dh0 + st : nullptr;
    const int wv = sc_wave();
    if (wv >= SC_NC) {
        if (w.q.nt > 0) sc_produce<OT, DK, DV, true>(a, w, (lds_char*)buf0, (lds_char*)buf1, wv - SC_NC);
        return;
    }
    sc_bwd_walk<OT, DK, DV>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
}

template <class OT, int DK, int DV>
hipError_t launch_sc_fwd_chain_t(const ScArgs& a, bool train, hipStream_t stream) {
    const dim3 grid((unsigned)(a.N * a.Hv * (DV / 16))), block(64 * (SC_NC + SC_NP));
    if (train && a.o)
        hipLaunchKernelGGL((k_sc_fwd_chain<OT, DK, DV, true, true>), grid, block, 0, stream, a);
    else if (train)
        hipLaunchKernelGGL((k_sc_fwd_chain<OT, DK, DV, true, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((k_sc_fwd_chain<OT, DK, DV, false, true>), grid, block, 0, stream, a);
    return hipGetLastError();
}
template <class OT, int DK, int DV>
hipError_t launch_sc_bwd_chain_t(const ScArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.N * a.Hv * (DV / 16))), block(64 * (SC_NC + SC_NP));
    hipLaunchKernelGGL((k_sc_bwd_chain<OT, DK, DV>), grid, block, 0, stream, a);
    return hipGetLastError();
}

#define GDR2_SC_CHAIN(OT_, DK_, DV_)                                                              \
    template hipError_t launch_sc_fwd_chain_t<OT_, DK_, DV_>(const ScArgs&, bool, hipStream_t);   \
    template hipError_t launch_sc_bwd_chain_t<OT_, DK_, DV_>(const ScArgs&, hipStream_t);
GDR2_SC_CHAIN(bf16, 64, 64)
GDR2_SC_CHAIN(bf16, 64, 128)
GDR2_SC_CHAIN(bf16, 128, 64)
GDR2_SC_CHAIN(bf16, 128, 128)
GDR2_SC_CHAIN(float, 64, 64)
#undef GDR2_SC_CHAIN

}  // namespace gdr2
