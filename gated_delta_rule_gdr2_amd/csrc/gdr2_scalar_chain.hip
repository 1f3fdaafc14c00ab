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
__device__ __forceinline__ void sc_dma(const char* src, lds_char* dst, int pi) {
    static_assert(BYTES % (1024 * SC_NP) == 0, "the same number of whole kilobytes for each producer");
    const unsigned lo = lane_id() * 16;
    src += pi * 1024;
    dst += pi * 1024;
#pragma unroll
    for (int k = 0; k < BYTES / 1024; k += SC_NP)
        __builtin_amdgcn_global_load_lds(src + k * 1024 + lo, (lds_void*)(dst + k * 1024), 16, 0, 0);
}
// ... of the 64 rows of a row-major tensor (row stride rs bytes, RL elements read of each) into a
// swizzled tile. A lane's place in a row group, swizzle included, repeats every 16 rows, so the lane
// part of the addresses is computed once (RowLanes) and a copy costs an addition to a scalar base:
// the producers' time is issue time, and with addresses computed copy by copy they held up the step.
// Rows from nvalid on repeat the last valid one: every product multiplies them by rows of beta, tail,
// e^gam, M or Delta that are exact zeros, and a caller's padding is not read.
template <class OT, int RL>
struct RowLanes {
    static constexpr int EPC = 16 / (int)sizeof(OT), NCH = RL / EPC, RPI = 64 / NCH, NP16 = 16 / RPI;
    unsigned off[NP16];  // row group n % NP16: byte offset of the lane's piece from the group's first row
    __device__ __forceinline__ RowLanes(size_t rs) {
        const int l = lane_id();
#pragma unroll
        for (int n = 0; n < NP16; ++n)
            off[n] = (unsigned)(l / NCH * rs) + ((l % NCH) ^ swz_f<OT, RL>(n * RPI + l / NCH)) * 16;
    }
};
template <class OT, int RL>
__device__ __forceinline__ void sc_dma_rows(const RowLanes<OT, RL>& rl, const char* base, size_t rs, int nvalid,
                                            lds_char* tile, int pi) {
    using R = RowLanes<OT, RL>;
    static_assert((CH / R::RPI) % SC_NP == 0 && R::NP16 % SC_NP == 0, "row groups split evenly");
    if (nvalid == CH) {
#pragma unroll
        for (int n = 0; n < CH / R::RPI; n += SC_NP) {
            // row group n + pi: its lane pattern is off[(n + pi) % NP16]
            const unsigned o = pi == 0 ? rl.off[n % R::NP16] : rl.off[(n + 1) % R::NP16];
            const char* src = base + (size_t)(n + pi) * R::RPI * rs + o;
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(tile + (n + pi) * 1024), 16, 0, 0);
        }
    } else {
        const int l = lane_id();
#pragma unroll 1
        for (int n = pi; n < CH / R::RPI; n += SC_NP) {
            const int row = n * R::RPI + l / R::NCH;
            const char* src = base + (size_t)min(row, nvalid - 1) * rs + ((l % R::NCH) ^ swz_f<OT, RL>(row)) * 16;
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(tile + n * 1024), 16, 0, 0);
        }
    }
}
// ... of a 16-column slice of the 64 rows, as [64][16]
template <class OT>
__device__ __forceinline__ void sc_dma_slice(const char* base, size_t rs, int nvalid, lds_char* tile, int pi) {
    constexpr int LPR = (int)sizeof(OT), RPI = 64 / LPR;  // 16-byte pieces of a row
    const int l = lane_id();
#pragma unroll
    for (int n = 0; n < CH / RPI; n += SC_NP) {
        const int row = min((n + pi) * RPI + l / LPR, nvalid - 1);
        __builtin_amdgcn_global_load_lds(base + (size_t)row * rs + l % LPR * 16, (lds_void*)(tile + (n + pi) * 1024),
                                         16, 0, 0);
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
    static constexpr int T = V + CH * 16 * ES;        // backward: NS images of T and of M
    static constexpr int M = T + (BWD ? NS : 0) * SQ;
    static constexpr int VEC = M + (BWD ? NS : 0) * SQ;
    static constexpr int BYTES = VEC + 2048;          // SC_VEC floats, in whole kilobytes
    static constexpr int F = xfrag<OT>();
    static constexpr int XS = 0;                      // state slice: NS x NKB fragments
    static constexpr int XX = XS + NS * NKB * F;      // X or dDelta: NS x 2
    static constexpr int XD = XX + NS * 2 * F;        // tail Delta or beta e^gam dY: NS x 2
    static constexpr int XO = XD + NS * 2 * F;        // Delta or dY, one part: 2
    static constexpr int XBYTES = XO + 2 * F;
    static_assert(2 * BYTES + XBYTES + 256 <= 160 * 1024, "two operand buffers fit");
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
__device__ __forceinline__ void sc_produce(const ScArgs& a, const ScWalk<OT>& w, lds_char* b0, lds_char* b1,
                                           lds_char* pf, int pi) {
    using B = ScChainLds<OT, DK, BWD>;
    const int nt = w.q.nt;
    const size_t rsk = (size_t)a.Hk * DK, rsv = (size_t)a.Hv * DV;
    const RowLanes<OT, DK> rl(rsk * B::ES);
    // the operands of chunk index(n), in two parts: k, v (dO), the row factors and T; q and M
    auto load1 = [&](int n) {
        const int c = BWD ? nt - 1 - n : n;
        lds_char* buf = (n & 1) ? b1 : b0;
        const long long row0 = w.q.tok0 + 64LL * c;
        const int nvalid = min(CH, w.q.len - CH * c);
        const size_t id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        sc_dma_rows<OT, DK>(rl, (const char*)((const OT*)a.k + row0 * rsk + (size_t)w.hk * DK), rsk * B::ES, nvalid,
                            buf + B::K, pi);
        const OT* v = BWD ? (const OT*)a.dout : (const OT*)a.v;
        sc_dma_slice<OT>((const char*)(v + row0 * rsv + (size_t)w.h * DV + 16 * w.j), rsv * B::ES, nvalid, buf + B::V,
                         pi);
        // the row factors: 1.5 KB of the 2 KB the buffer has for them
        const char* src = a.ws + a.L.o_vec + id * a.L.vec * 4;
        const unsigned lo = (pi == 0 ? lane_id() : 64 + (lane_id() & 31)) * 16;
        __builtin_amdgcn_global_load_lds(src + lo, (lds_void*)(buf + B::VEC + pi * 1024), 16, 0, 0);
        if constexpr (BWD) sc_dma<B::NS * B::SQ>(a.ws + a.L.o_t + id * a.L.t * B::ES, buf + B::T, pi);
    };
    auto load2 = [&](int n) {
        if (!BWD && !a.o) return;
        const int c = BWD ? nt - 1 - n : n;
        lds_char* buf = (n & 1) ? b1 : b0;
        const long long row0 = w.q.tok0 + 64LL * c;
        const int nvalid = min(CH, w.q.len - CH * c);
        const size_t id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        sc_dma_rows<OT, DK>(rl, (const char*)((const OT*)a.q + row0 * rsk + (size_t)w.hk * DK), rsk * B::ES, nvalid,
                            buf + B::Q, pi);
        if constexpr (BWD) sc_dma<B::NS * B::SQ>(a.ws + a.L.o_m + id * a.L.m * B::ES, buf + B::M, pi);
    };
    // L2 prefetch of chunk index(n): one word of every 128-byte line of its operands, into a word of
    // LDS that nothing reads. The lines are numbered 0 .. LINES - 1 over k, T, [q, M,] v (dO) and the row
    // factors, and shared between the NJ slices of the (sequence, head), which sit on one L2.
    constexpr int ES = B::ES, NJ = DV / 16;
    constexpr int LPK = DK * ES / 128, LPV = DV * ES / 128;  // lines of a row
    constexpr int LK = CH * LPK, LT = B::NS * B::SQ / 128, LM = (BWD ? B::NS : 1) * B::SQ / 128, LV = CH * LPV;
    constexpr int LVEC = SC_VEC * 4 / 128, LINES = 2 * LK + LT + LM + LV + LVEC;
    constexpr int NPF = (LINES + NJ * 64 * SC_NP - 1) / (NJ * 64 * SC_NP);
    auto prefetch = [&](int n) {  // (past the last chunk: the last one again, so that their number is fixed)
        n = min(n, nt - 1);
        const int c = BWD ? nt - 1 - n : n;
        const long long row0 = w.q.tok0 + 64LL * c;
        const int last = min(CH, w.q.len - CH * c) - 1;
        const size_t id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        const char* kp = (const char*)((const OT*)a.k + row0 * rsk + (size_t)w.hk * DK);
        const char* qp = (const char*)((const OT*)a.q + row0 * rsk + (size_t)w.hk * DK);
        const char* vp = (const char*)((BWD ? (const OT*)a.dout : (const OT*)a.v) + row0 * rsv + (size_t)w.h * DV);
        const char* tp = a.ws + a.L.o_t + id * a.L.t * ES;
        const char* mp = a.ws + a.L.o_m + id * a.L.m * ES;
        const char* fp = a.ws + a.L.o_vec + id * a.L.vec * 4;
#pragma unroll
        for (int i = 0; i < NPF; ++i) {
            int v = ((i * SC_NP + pi) * 64 + lane_id()) * NJ + w.j;
            const char* p;
            if (v < LK) {
                p = kp + (size_t)min(v / LPK, last) * rsk * ES + (v % LPK) * 128;
            } else if ((v -= LK) < LT) {
                p = tp + v * 128;
            } else if ((v -= LT) < LV) {
                p = vp + (size_t)min(v / LPV, last) * rsv * ES + (v % LPV) * 128;
            } else if ((v -= LV) < LK) {
                p = qp + (size_t)min(v / LPK, last) * rsk * ES + (v % LPK) * 128;
            } else if ((v -= LK) < LM) {
                p = mp + v * 128;
            } else {
                p = fp + min(v - LM, LVEC - 1) * 128;
            }
            __builtin_amdgcn_global_load_lds(p, (lds_void*)(pf), 4, 0, 0);
        }
    };
    constexpr int AHEAD = 3;  // chunks between a line's prefetch and its copy into LDS
    load1(0);
    load2(0);
    for (int n = 1; n <= AHEAD; ++n) prefetch(n);
    wait_vm<0>();
    for (int n = 0; n < nt; ++n) {
        sync_lds();  // A: chunk n is in its buffer; the other buffer (chunk n - 1) is free
        if (n + 1 < nt) load1(n + 1);
        sync_lds();  // B
        if (n + 1 < nt) load2(n + 1);
        sync_lds();  // C
        prefetch(n + 1 + AHEAD);
        wait_vm<NPF>();  // chunk n + 1 is in; this step's prefetch goes on
    }
    wait_vm<0>();  // no copy into this workgroup's LDS outlives it
}

// Compute waves: the products that lead from one state to the next, and nothing else. What a step
// reads from its operand buffer is read as early as the buffer allows (T and K^T behind the reads that
// the first product waits for), so that behind the barriers B and C only the exchanged fragments are
// left to wait for.
template <class OT, int DK, int DV>
__device__ __forceinline__ void sc_fwd_walk(const ScArgs& a, const ScWalk<OT>& w, int wv, lds_char* b0, lds_char* b1,
                                            lds_char* xs) {
    using B = ScChainLds<OT, DK, false>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F, NT = DK / 64;  // NT: 16-row state tiles of a wave
    const int l = lane_id(), li = l & 15, lq = l >> 4;
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
    // this wave's rows of T go from the workspace straight into registers, a step ahead
    const OT* tp = (const OT*)(a.ws + a.L.o_t) + ((size_t)w.q.slot0 * a.Hv + w.h) * a.L.t;
    const size_t tstep = (size_t)a.Hv * a.L.t;
    FT Tn[NS][2];
    auto load_t = [&]() {
#pragma unroll
        for (int p = 0; p < NS; ++p)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) Tn[p][kb] = gfrag_img<OT, CH>(tp + p * CH * CH, 16 * wv, 32 * kb);
    };
    if (nt > 0) load_t();
#pragma unroll 1
    for (int n = 0; n < nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vK{buf + B::K};
        sync_lds();  // A: the state slice is published, the chunk's operands are in
        FT SB[NS][NKB], Kf[NKB];
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            Kf[kb] = lfrag_rowk8<OT>(vK, 16 * wv, 32 * kb);
#pragma unroll
            for (int p = 0; p < NS; ++p) SB[p][kb] = get_x<OT>(xs + B::XS + (p * NKB + kb) * F);
        }
        float e4[4], b4[4], t4[4], v4[4];
        lds_get4<float>(buf + B::VEC + (SC_E + 16 * wv + 4 * lq) * 4, e4);
        lds_get4<float>(buf + B::VEC + (SC_BETA + 16 * wv + 4 * lq) * 4, b4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v4[i] = lds_get1<OT>(buf + B::V + ((16 * wv + 4 * lq + i) * 16 + li) * B::ES);
        lds_get4<float>(buf + B::VEC + (SC_TAIL + 16 * wv + 4 * lq) * 4, t4);
        const float ec = lds_load<float>(buf + B::VEC + SC_EC * 4);
        __builtin_amdgcn_sched_barrier(0);
        // X = beta (V - e^gam K S) on this wave's tokens
        f32x4 Y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int p = 0; p < NS; ++p) mma(Y[2 * (kb & 1) + p], Kf[kb], SB[p][kb]);
        Y[0] = (Y[0] + Y[2]) + (Y[1] + Y[3]);
        f32x4 X;
#pragma unroll
        for (int i = 0; i < 4; ++i) X[i] = b4[i] * (v4[i] - e4[i] * Y[0][i]);
        put_split<OT>(xs + B::XX + (wv >> 1) * F, 2 * F, wv & 1, X);
        sync_lds();  // B: X is published
        // Delta = T X on this wave's tokens (T is lower triangular: for token tiles 0 and 1 the second
        // half of the columns is zero)
        FT XB[NS][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int p = 0; p < NS; ++p) XB[p][kb] = get_x<OT>(xs + B::XX + (2 * p + kb) * F);
        FT KT[NT][2];  // K^T, rows: this wave's keys
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) KT[t][kb] = lfrag_colk8<OT>(vK, 16 * (NT * wv + t), 32 * kb);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 D[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) D[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int p = 0; p < NS; ++p)
#pragma unroll
                for (int r = 0; r < NS; ++r) mma(D[2 * p + r], Tn[r][kb], XB[p][kb]);
        if (n + 1 < nt) tp += tstep;  // (past the last chunk: the last again)
        load_t();
        D[0] = (D[0] + D[1]) + (D[2] + D[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) D[1][i] = t4[i] * D[0][i];
        put_split<OT>(xs + B::XD + (wv >> 1) * F, 2 * F, wv & 1, D[1]);
        put_one<OT>(xs + B::XO + (wv >> 1) * F, wv & 1, D[0]);
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
                mma(s0, KT[t][kb], DB[0][kb]);
                if constexpr (NS == 2) mma(s1, KT[t][kb], DB[1][kb]);
            }
            S[t] = s0 + s1;
        }
        publish_state();
    }
    if (w.end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w.end[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * DV + 16 * w.j + li] = S[t][i];
    }
}

// The 16-column slice [rows][16] of an exchanged matrix of 16 RT rows (its fragments' first parts, from
// frag on) to the workspace, by the four side waves.
template <class OT, int RT>
__device__ __forceinline__ void store_slice(const lds_char* frag, OT* dst, int wv) {
    if constexpr (sizeof(OT) == 2) {
#pragma unroll
        for (int t = 0; t < (RT + 3) / 4; ++t) {
            const int rt = wv + 4 * t;
            if (RT % 4 == 0 || rt < RT) store_slice_tr(frag + (rt >> 1) * xfrag<OT>(), rt & 1, dst + rt * 256);
        }
    } else {
        const int l = lane_id(), li = l & 15, lq = l >> 4;
        if (wv < RT / 2) {
            const auto f = get_x<OT>(frag + wv * xfrag<OT>());
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[(32 * wv + 8 * lq + e) * 16 + li] = f[e];
        }
    }
}

// Side waves: what a step gives away -- O, and for training the chunk's start state and Delta.
template <class OT, int DK, int DV, bool TRAIN, bool OUT>
__device__ __forceinline__ void sc_fwd_side(const ScArgs& a, const ScWalk<OT>& w, int wv, const lds_char* b0,
                                            const lds_char* b1, const lds_char* xs) {
    using B = ScChainLds<OT, DK, false>;
    using FT = typename Frag<OT>::type;
    constexpr int NKB = B::NKB, F = B::F;
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const OT* mp = (const OT*)(a.ws + a.L.o_m) + ((size_t)w.q.slot0 * a.Hv + w.h) * a.L.m;
    const size_t mstep = (size_t)a.Hv * a.L.m;
    FT M[2];  // this wave's rows of M, a step ahead as T in the compute waves
    auto load_m = [&]() {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) M[kb] = gfrag_img<OT, CH>(mp, 16 * wv, 32 * kb);
    };
    if (OUT && w.q.nt > 0) load_m();
#pragma unroll 1
    for (int n = 0; n < w.q.nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const size_t id = (size_t)(w.q.slot0 + n) * a.Hv + w.h;
        sync_lds();  // A
        sync_lds();  // B: from here to C the compute waves leave LDS mostly idle
        // O^T (rows: value columns, columns: this wave's tokens), the state's part
        f32x4 O = {0.f, 0.f, 0.f, 0.f};
        if (OUT) {
            const LSwz<OT, DK> vQ{buf + B::Q};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) mma(O, get_x<OT>(xs + B::XS + kb * F), lfrag_rowk8<OT>(vQ, 16 * wv, 32 * kb));
            O = O * lds_load<float>(buf + B::VEC + (SC_E + 16 * wv + li) * 4);
        }
        if (TRAIN) store_slice<OT, DK / 16>(xs + B::XS, (OT*)(a.ws + a.L.o_s) + id * a.L.s + (size_t)w.j * DK * 16, wv);
        sync_lds();  // C
        if (OUT) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) mma(O, get_x<OT>(xs + B::XO + kb * F), M[kb]);
            if (n + 1 < w.q.nt) mp += mstep;
            load_m();
            const int row = 16 * wv + li;
            if (CH * n + row < w.q.len) {
                const float ov[4] = {O[0], O[1], O[2], O[3]};
                st4((OT*)a.o + ((size_t)(w.q.tok0 + 64LL * n + row) * a.Hv + w.h) * DV + 16 * w.j + 4 * lq, ov);
            }
        }
        if (TRAIN) store_slice<OT, 4>(xs + B::XO, (OT*)(a.ws + a.L.o_delta) + id * a.L.d + (size_t)w.j * CH * 16, wv);
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
__global__ __launch_bounds__(64 * (2 * SC_NC + SC_NP)) void k_sc_fwd_chain(ScArgs a) {
    using B = ScChainLds<OT, DK, false>;
    __shared__ __align__(16) char buf0[B::BYTES];
    __shared__ __align__(16) char buf1[B::BYTES];
    __shared__ __align__(16) char xch[B::XBYTES];
    __shared__ __align__(16) char pfslot[256];  // target of the prefetches, never read
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
    if (wv < SC_NC)
        sc_fwd_walk<OT, DK, DV>(a, w, wv, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (wv < 2 * SC_NC)
        sc_fwd_side<OT, DK, DV, TRAIN, OUT>(a, w, wv - SC_NC, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (w.q.nt > 0)
        sc_produce<OT, DK, DV, false>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)pfslot, wv - 2 * SC_NC);
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
    __shared__ __align__(16) char pfslot[256];  // target of the prefetches, never read
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
        if (w.q.nt > 0) sc_produce<OT, DK, DV, true>(a, w, (lds_char*)buf0, (lds_char*)buf1,
                                                   (lds_char*)pfslot, wv - SC_NC);
        return;
    }
    sc_bwd_walk<OT, DK, DV>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
}

template <class OT, int DK, int DV>
hipError_t launch_sc_fwd_chain_t(const ScArgs& a, bool train, hipStream_t stream) {
    const dim3 grid((unsigned)(a.N * a.Hv * (DV / 16))), block(64 * (2 * SC_NC + SC_NP));
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
