// Gated delta rule with scalar gates: the two sequential chains (equations in gdr2_scalar.hpp).
//
//   forward  : Y = K S ;  X = beta (V - e^gam Y) ;  Delta = T X ;
//              O = e^gam Q S + M Delta ;  S' = e^gamC S + K^T (tail Delta)
//   backward : dDelta = M^T dO + tail K dS' ;  dY = T^T dDelta ;
//              dS = e^gamC dS' + Q^T (e^gam dO) - K^T (beta e^gam dY)
//
// Each (sequence, value head, 16 value columns) is its own chain over the chunks, and a workgroup walks
// one or two of them (sc_column_tiles): four compute waves, four side waves and two producer waves. Compute
// wave w owns token tile w and d_k / 4 key rows of the state slice, which stay in fp32 accumulators for the
// whole walk. A step is three products that follow one another, with the intermediate published through
// LDS between them (barriers A, B, C): the state slice, X (dDelta), and tail Delta (beta e^gam dY).
// Everything that reaches the state goes through as NS parts (Split in gdr2_scalar_device.hpp): the state
// and its gradient come out to about 5e-6, at two to four bf16 products for one, on matrix cores that wait
// for operands most of the time anyway. What a step gives away (O, and for training the states, Delta and
// dY) or what does not depend on the state (Q^T (e^gam dO)) is the side waves', between the same barriers.
//
// Against the chains of the channel-wise operator, which read five per-chunk matrices that their
// intra-chunk kernel wrote (W_m, K_d^T, Q_g, M, U), these read the caller's own q, k, v and T, M:
// the scalar decay scales accumulators instead of operands, so K S and K^T Delta share one raw K tile
// in LDS (read by rows and, transposed, by columns), and value heads that share a key head share
// its rows in L2.
//
// The producers stream k, q, v (dO) and the row factors of a chunk into LDS by asynchronous DMA, 16 bytes a
// lane, into two buffers, the next chunk's while this one's step runs, and call what the workgroups of a head
// will read three chunks later into their L2, each a share of it. T and M go from L2 straight to registers.
//
// Few long sequences are cut in segments (sc_segments): the state at a segment's end is affine in the one at
// its start, E + P S, and one launch finds E and P of all segments with the same walk (SUM: P from the unit
// matrix, with the values counted as zero), k_sc_join carries them forward, and the walks proper start from
// there. (With 64 walks and more the first segment is walked in full at once: ScArgs::lead.)
//
// Bound by the latency of a step: 256 walks of 64 steps (2 x 4096 tokens, 16 heads, d = 128, one walk on each
// compute unit) take 96 us forward with what training saves and 101 us backward, 1.5 us a step; 128 walks
// of 256 steps (one prompt of 16384 tokens, walked whole) 283 us, 1.1 us or 2700 cycles a step, of which the three
// barriers with the exchange behind each are most. Measured and not taken: T through LDS like the rest
// (forward 104 -> 111 us at the time), q straight to the side waves' registers (104 -> 113), the keys of K S
// split over the waves and summed through LDS (97 -> 108; the prompt 288 -> 333), a higher wave priority
// for the compute waves (no change).
#include <type_traits>

#include "gdr2_intra_common.hpp"
#include "gdr2_scalar_device.hpp"

namespace gdr2 {

constexpr int SC_NC = 4;  // compute waves
constexpr int SC_NP = 2;  // producer waves

__device__ __forceinline__ int sc_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Producer pi's share of a copy of the 64 rows of a row-major tensor (row stride rs bytes, RL elements of each) into a
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
// their number allows. even: walks of one length, so that an XCD may take consecutive ones (uneven ones
// come longest first, and that order is kept)
__device__ __forceinline__ void sc_chain_map(int gid, int pairs, int NJ, bool even, int& s, int& j) {
    const int x = gid % 8, rest = gid / 8;
    if (pairs % 8 == 0) {
        j = rest % NJ;
        s = (rest / NJ) * 8 + x;
    } else if (even) {
        const int all = pairs * NJ, n = x * (all / 8) + min(x, all % 8) + rest;
        s = n / NJ;
        j = n % NJ;
    } else {
        s = gid / NJ;
        j = gid % NJ;
    }
}

// NC: 16-column tiles of the value axis a workgroup walks
template <class OT, int DK, int NC, bool BWD>
struct ScChainLds {  // one operand buffer, and the exchange
    static constexpr int ES = sizeof(OT), NS = Split<OT>::NS, NKB = DK / 32;
    static constexpr int K = 0;
    static constexpr int Q = K + CH * DK * ES;
    static constexpr int V = Q + CH * DK * ES;        // v (forward) or dO (backward), NC tiles [64][16]
    static constexpr int VT = CH * 16 * ES;
    static constexpr int VEC = V + NC * VT;
    static constexpr int BYTES = VEC + 2048;          // SC_VEC floats, in whole kilobytes
    static constexpr int F = xfrag<OT>();
    // exchange, for each column tile
    static constexpr int XS = 0;                      // state: NS x NKB fragments
    static constexpr int XX = XS + NS * NKB * F;      // X or dDelta: NS x 2
    static constexpr int XD = XX + NS * 2 * F;        // tail Delta or -beta e^gam dY: NS x 2
    static constexpr int XO = XD + NS * 2 * F;        // Delta: NS x 2; dY, one part: 2
    static constexpr int XP = XO + (BWD ? 1 : NS) * 2 * F;  // backward: Q^T (e^gam dO), fp32 accumulator tiles
    static constexpr int XT = XP + (BWD ? DK / 16 * 1024 : 0);
    static constexpr int XBYTES = NC * XT;
    static_assert(2 * BYTES + XBYTES + 256 <= 160 * 1024, "two operand buffers fit");
};

// Where a walk finds its data; j: its workgroup among those of the (sequence, value head). Its states are
// columns col .. of matrices with ld columns; unit: it starts from those columns of the unit matrix, and the
// values (dO) count as zero. full: what its steps give away is wanted, not only where it ends.
struct ScWalk {
    ScSeq q;
    int h, hk, j, ld, col;
    bool unit, full;
    const float* start;
    float* end;
};

// A producer's side: the operands of chunk index(n), n = 0 .. nt - 1, into buffer n % 2. Takes part
// in the step's barriers.
// (FULL: backward, and forward with outputs, which alone read q and M; with SUM, of full walks.)
template <class OT, int DK, int DV, int NC, bool BWD, bool FULL, bool SUM>
__device__ __forceinline__ void sc_produce(const ScArgs& a, const ScWalk& w, lds_char* b0, lds_char* b1, lds_char* pf,
                                           int pi) {
    using B = ScChainLds<OT, DK, NC, BWD>;
    constexpr int ES = B::ES, NJ = DV / (16 * NC);
    const int nt = w.q.nt;
    const size_t rsk = (size_t)a.Hk * DK * ES, rsv = (size_t)a.Hv * DV * ES;  // row strides, bytes
    const RowLanes<OT, DK> rl(rsk);
    struct Chunk {
        const char *k, *q, *v, *f;
        int nvalid;
        size_t id;
    };
    auto chunk = [&](int n) {
        const int c = BWD ? nt - 1 - n : n;
        const long long row0 = w.q.tok0 + 64LL * c;
        Chunk x;
        x.nvalid = min(CH, w.q.len - CH * c);
        x.id = (size_t)(w.q.slot0 + c) * a.Hv + w.h;
        x.k = (const char*)a.k + row0 * rsk + (size_t)w.hk * DK * ES;
        x.q = (const char*)a.q + row0 * rsk + (size_t)w.hk * DK * ES;
        x.v = (const char*)(BWD ? a.dout : a.v) + row0 * rsv + (size_t)w.h * DV * ES;
        x.f = a.ws + a.L.o_vec + x.id * a.L.vec * 4;
        return x;
    };
    auto load1 = [&](int n) {  // k, v (dO) and the row factors
        const Chunk x = chunk(n);
        lds_char* buf = (n & 1) ? b1 : b0;
        sc_dma_rows<OT, DK>(rl, x.k, rsk, x.nvalid, buf + B::K, pi);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
            sc_dma_slice<OT>(x.v + 16 * (NC * w.j + ch) * ES, rsv, x.nvalid, buf + B::V + ch * B::VT, pi);
        // the row factors: 1.5 KB of the 2 KB the buffer has for them
        const unsigned lo = (pi == 0 ? lane_id() : 64 + (lane_id() & 31)) * 16;
        const char* src = x.f + lo;
        __builtin_amdgcn_global_load_lds(src, (lds_void*)(buf + B::VEC + pi * 1024), 16, 0, 0);
    };
    auto load2 = [&](int n) {  // q
        if (!FULL || (SUM && !BWD && !w.full)) return;
        const Chunk x = chunk(n);
        sc_dma_rows<OT, DK>(rl, x.q, rsk, x.nvalid, ((n & 1) ? b1 : b0) + B::Q, pi);
    };
    // L2 prefetch of chunk index(n): one word of every 128-byte line of what the workgroup reads of it,
    // into a word of LDS that nothing reads. The lines are numbered over k, T, v (dO), q, M and the row
    // factors, and shared between the NJ workgroups of the (sequence, head), which sit on one L2.
    constexpr int LPK = DK * ES / 128, LPV = DV * ES / 128;  // lines of a row
    constexpr int LF = 512 * ES / 128;                       // of an image's fragment, six of eight to read
    constexpr int LK = CH * LPK, LT = B::NS * 6 * LF, LM = (BWD ? B::NS : 1) * 6 * LF, LV = CH * LPV;
    auto img_line = [](int v) {
        const int p = v / (6 * LF), f = v / LF % 6;
        return (8 * p + (BWD ? (f < 4 ? f : 2 * f - 3) : (f < 2 ? 2 * f : f + 2))) * LF + v % LF;
    };
    constexpr int LVEC = SC_VEC * 4 / 128, LINES = LK + LT + LV + (FULL ? LK + LM : 0) + LVEC;
    constexpr int NPF = (LINES + NJ * 64 * SC_NP - 1) / (NJ * 64 * SC_NP);
    auto prefetch = [&](int n) {  // (past the last chunk: the last one again, so that their number is fixed)
        const Chunk x = chunk(min(n, nt - 1));
        const int last = x.nvalid - 1;
        const char* tp = a.ws + (BWD ? a.L.o_tt : a.L.o_t) + x.id * a.L.t * ES;
        const char* mp = a.ws + (BWD ? a.L.o_mt : a.L.o_m) + x.id * (BWD ? a.L.t : a.L.m) * ES;
#pragma unroll
        for (int i = 0; i < NPF; ++i) {
            int v = ((i * SC_NP + pi) * 64 + lane_id()) * NJ + w.j;
            const char* p;
            if (v < LK) {
                p = x.k + (size_t)min(v / LPK, last) * rsk + (v % LPK) * 128;
            } else if ((v -= LK) < LT) {
                p = tp + img_line(v) * 128;
            } else if ((v -= LT) < LV) {
                p = x.v + (size_t)min(v / LPV, last) * rsv + (v % LPV) * 128;
            } else if (FULL && SUM && !BWD && !w.full) {
                p = x.f + min(max(v - LV - LK - LM, 0), LVEC - 1) * 128;
            } else if (FULL && (v -= LV) < LK) {
                p = x.q + (size_t)min(v / LPK, last) * rsk + (v % LPK) * 128;
            } else if (FULL && (v -= LK) < LM) {
                p = mp + img_line(v) * 128;
            } else {
                p = x.f + min(v - (FULL ? LM : LV), LVEC - 1) * 128;
            }
            __builtin_amdgcn_global_load_lds(p, (lds_void*)(pf), 4, 0, 0);
        }
    };
    constexpr int AHEAD = 3;  // chunks between a line's prefetch and its use
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

// A wave's 16 rows of a pair of [64][64] triangular images (TR: upper), straight from the workspace into
// registers: the fragments are whole kilobytes there, each read by one wave, and would pass LDS twice for
// nothing. Of the eight, the two above (below) the diagonal are not read.
template <class OT, int NS, bool TR>
struct ImgRows {
    typename Frag<OT>::type f[NS][2];
    __device__ __forceinline__ void load(const OT* p, int wv) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (sc_img_zero<TR>(wv, kb))
                    f[n][kb] = {};
                else
                    f[n][kb] = gfrag_img<OT, CH>(p + n * CH * CH, 16 * wv, 32 * kb);
    }
};

// One wave's tiles of a state slice: tile t of column tile ch holds key rows 16 (NT wv + t) + 4 lq + i,
// column 16 ch + li of the walk's columns.
template <class OT, int DK, int NC, bool BWD>
struct ScState {
    using B = ScChainLds<OT, DK, NC, BWD>;
    static constexpr int NT = DK / 64;
    f32x4 s[NC][NT];
    __device__ __forceinline__ void init(const ScWalk& w, int wv) {
        const int l = lane_id(), li = l & 15, lq = l >> 4;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * (NT * wv + t) + 4 * lq + i, c = w.col + 16 * ch + li;
                    s[ch][t][i] = w.unit ? (r == c ? 1.f : 0.f) : w.start ? w.start[(size_t)r * w.ld + c] : 0.f;
                }
    }
    __device__ __forceinline__ void out(const ScWalk& w, int wv) const {
        const int l = lane_id(), li = l & 15, lq = l >> 4;
        if (!w.end) return;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w.end[(size_t)(16 * (NT * wv + t) + 4 * lq + i) * w.ld + w.col + 16 * ch + li] = s[ch][t][i];
    }
    __device__ __forceinline__ void publish(lds_char* xs, int ch, int wv) const {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int rt = NT * wv + t;
            put_split<OT>(xs + ch * B::XT + B::XS + (rt >> 1) * B::F, B::NKB * B::F, rt & 1, s[ch][t]);
        }
    }
};

// Compute waves: the products that lead from one state to the next, and nothing else. What a step
// reads from its operand buffer is read as early as the buffer allows (K^T behind the reads that the
// second product waits for), so that behind the barrier C only the exchanged fragments are left to
// wait for.
template <class OT, int DK, int DV, int NC, bool SUM>
__device__ __forceinline__ void sc_fwd_walk(const ScArgs& a, const ScWalk& w, int wv, lds_char* b0, lds_char* b1,
                                            lds_char* xs) {
    using B = ScChainLds<OT, DK, NC, false>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F, NT = DK / 64;
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const int nt = w.q.nt;
    ScState<OT, DK, NC, false> S;
    S.init(w, wv);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) S.publish(xs, ch, wv);
    const OT* tp = (const OT*)(a.ws + a.L.o_t) + ((size_t)w.q.slot0 * a.Hv + w.h) * a.L.t;
    const size_t tstep = (size_t)a.Hv * a.L.t;
    ImgRows<OT, NS, false> T;  // a step ahead
    if (nt > 0) T.load(tp, wv);
#pragma unroll 1
    for (int n = 0; n < nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vK{buf + B::K};
        sync_lds();  // A: the state slice is published, the chunk's operands are in
        // X = beta (V - e^gam K S) on this wave's tokens
        FT Kf[NKB];
        float e4[4], b4[4], t4[4];
        lds_get4<float>(buf + B::VEC + (SC_E + 16 * wv + 4 * lq) * 4, e4);
        lds_get4<float>(buf + B::VEC + (SC_BETA + 16 * wv + 4 * lq) * 4, b4);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            lds_char* xc = xs + ch * B::XT;
            FT SB[NS][NKB];
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                if (ch == 0) Kf[kb] = lfrag_rowk8<OT>(vK, 16 * wv, 32 * kb);
#pragma unroll
                for (int p = 0; p < NS; ++p) SB[p][kb] = get_x<OT>(xc + B::XS + (p * NKB + kb) * F);
            }
            float v4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v4[i] = lds_get1<OT>(buf + B::V + ch * B::VT + ((16 * wv + 4 * lq + i) * 16 + li) * B::ES);
            __builtin_amdgcn_sched_barrier(0);
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
            for (int i = 0; i < 4; ++i) X[i] = b4[i] * ((SUM && w.unit ? 0.f : v4[i]) - e4[i] * Y[0][i]);
            put_split<OT>(xc + B::XX + (wv >> 1) * F, 2 * F, wv & 1, X);
        }
        lds_get4<float>(buf + B::VEC + (SC_TAIL + 16 * wv + 4 * lq) * 4, t4);
        const float ec = lds_load<float>(buf + B::VEC + SC_EC * 4);
        sync_lds();  // B: X is published
        // Delta = T X on this wave's tokens
        FT KT[NT][2];  // K^T, rows: this wave's keys
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            lds_char* xc = xs + ch * B::XT;
            FT XB[NS][2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p) XB[p][kb] = get_x<OT>(xc + B::XX + (2 * p + kb) * F);
            if (ch == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) KT[t][kb] = lfrag_colk8<OT>(vK, 16 * (NT * wv + t), 32 * kb);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 D[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) D[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p)
#pragma unroll
                    for (int r = 0; r < NS; ++r) mma(D[2 * p + r], T.f[r][kb], XB[p][kb]);
            D[0] = (D[0] + D[1]) + (D[2] + D[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) D[1][i] = t4[i] * D[0][i];
            put_split<OT>(xc + B::XD + (wv >> 1) * F, 2 * F, wv & 1, D[1]);
            put_split<OT>(xc + B::XO + (wv >> 1) * F, 2 * F, wv & 1, D[0]);
        }
        sync_lds();  // C: Delta is published
        // the next T: from here to A the memory path is least busy, and a wave waits where it issues a load
        if (n + 1 < nt) tp += tstep;  // (past the last chunk: the last again)
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            const lds_char* xc = xs + ch * B::XT;
            FT DB[NS][2];
#pragma unroll
            for (int p = 0; p < NS; ++p)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) DB[p][kb] = get_x<OT>(xc + B::XD + (2 * p + kb) * F);
            if (ch == 0) T.load(tp, wv);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 s0 = S.s[ch][t] * ec, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    mma(s0, KT[t][kb], DB[0][kb]);
                    if constexpr (NS == 2) mma(s1, KT[t][kb], DB[1][kb]);
                }
                S.s[ch][t] = s0 + s1;
            }
            S.publish(xs, ch, wv);
        }
    }
    S.out(w, wv);
}

// The 16-column slice [rows][16] of an exchanged matrix of 16 RT rows (its fragments' first parts, from
// frag on) to the workspace, by the four side waves: read while the exchange holds it, stored later, since
// a wave waits where it issues a store and the others then wait for it at the next barrier. What is saved for
// the gradients (S, dS', Delta, dY) is one bf16 each: the gradients end in bf16, off by 2.3 to 2.9e-3, and a second
// part would add half as much again to the 208 KB a chunk and head that their kernel waits for. The chains
// themselves carry both parts on.
template <class OT, int RT>
struct Slice {
    static constexpr int N = sizeof(OT) == 2 ? (RT + 3) / 4 : 2;
    typename Raw4<OT>::type x[N];
    __device__ __forceinline__ void read(const lds_char* frag, int wv) {
        if constexpr (sizeof(OT) == 2) {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int rt = wv + 4 * t;
                if (RT % 4 == 0 || rt < RT) x[t] = read_slice_tr(frag + (rt >> 1) * xfrag<OT>(), rt & 1);
            }
        } else if (wv < RT / 2) {
            const lds_char* p = frag + wv * xfrag<OT>() + lane_id() * 32;
            x[0] = lds_load<f32x4>(p);
            x[1] = lds_load<f32x4>(p + 16);
        }
    }
    __device__ __forceinline__ void write(OT* dst, int wv) const {
        const int l = lane_id(), li = l & 15, lq = l >> 4;
        if constexpr (sizeof(OT) == 2) {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int rt = wv + 4 * t;
                if (RT % 4 == 0 || rt < RT) store_out<true>((bf16x4*)(dst + rt * 256 + li * 16 + 4 * lq), x[t]);
            }
        } else if (wv < RT / 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[(32 * wv + 8 * lq + e) * 16 + li] = x[e / 4][e % 4];
        }
    }
};

// Side waves: what a step gives away -- O, and for training the chunk's start state and Delta. In bf16 each of
// O's terms is off by one rounding, S's first part in one and M in the other, and O by its own: 2.4e-3 together
// (its own alone 1.7e-3). Delta has both parts: with one it was 2.9e-3. With both parts of S and M too it was
// 1.65e-3, and a prompt of 16384 tokens took 357 us instead of 322, a training step of 2 x 4096 345 instead of
// 331. M Delta is added, and O stored, behind the next chunk's barrier A, where nothing waits for these waves: in
// the step itself the prompt took 335 us. In training, where the chunk's state is stored there, it is the other
// way round: 346 us behind A, 334 in the step.
template <class OT, int DK, int DV, int NC, bool TRAIN, bool OUT, bool SUM>
__device__ __forceinline__ void sc_fwd_side(const ScArgs& a, const ScWalk& w, int wv, const lds_char* b0,
                                            const lds_char* b1, const lds_char* xs) {
    if (SUM && !w.full) {
#pragma unroll 1
        for (int n = 0; n < 3 * w.q.nt; ++n) sync_lds();  // A, B, C
        return;
    }
    using B = ScChainLds<OT, DK, NC, false>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F;
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    const OT* mp = (const OT*)(a.ws + a.L.o_m) + ((size_t)w.q.slot0 * a.Hv + w.h) * a.L.m;
    const size_t mstep = (size_t)a.Hv * a.L.m;
    ImgRows<OT, 1, false> M;  // a step ahead
    if (OUT && w.q.nt > 0) M.load(mp, wv);
    Slice<OT, DK / 16> S[NC];
    auto store_state = [&](int n) {  // chunk n's start state
        OT* p = (OT*)(a.ws + a.L.o_s) + ((size_t)(w.q.slot0 + n) * a.Hv + w.h) * a.L.s;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) S[ch].write(p + (size_t)(NC * w.j + ch) * DK * 16, wv);
    };
    f32x4 O[NC];  // O^T (rows: value columns, columns: this wave's tokens)
    auto finish = [&](int n) {  // chunk n's M Delta, and its rows of O
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p)
                    mma(O[ch], get_x<OT>(xs + ch * B::XT + B::XO + (2 * p + kb) * F), M.f[0][kb]);
        if (n + 1 < w.q.nt) mp += mstep;
        M.load(mp, wv);
        const int row = 16 * wv + li;
        if (CH * n + row < w.q.len) {
            OT* o = (OT*)a.o + ((size_t)(w.q.tok0 + 64LL * n + row) * a.Hv + w.h) * DV + 16 * NC * w.j + 4 * lq;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                const float ov[4] = {O[ch][0], O[ch][1], O[ch][2], O[ch][3]};
                st4(o + 16 * ch, ov);
            }
        }
    };
    constexpr bool LATE = OUT && !TRAIN;
#pragma unroll 1
    for (int n = 0; n < w.q.nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const size_t id = (size_t)(w.q.slot0 + n) * a.Hv + w.h;
        sync_lds();  // A
        if (LATE && n > 0) finish(n - 1);  // (until the next barrier the exchange still holds its Delta)
        if (TRAIN && n > 0) store_state(n - 1);
        FT Q[NKB];
        if (OUT) {
            const LSwz<OT, DK> vQ{buf + B::Q};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) Q[kb] = lfrag_rowk8<OT>(vQ, 16 * wv, 32 * kb);
        }
        sync_lds();  // B: from here to C the compute waves leave LDS mostly idle
        if (OUT) {  // O, the state's part
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) O[ch] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int ch = 0; ch < NC; ++ch) mma(O[ch], get_x<OT>(xs + ch * B::XT + B::XS + kb * F), Q[kb]);
            const float e = lds_load<float>(buf + B::VEC + (SC_E + 16 * wv + li) * 4);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) O[ch] = O[ch] * e;
        }
        if (TRAIN) {
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) S[ch].read(xs + ch * B::XT + B::XS, wv);
        }
        sync_lds();  // C
        if (OUT && !LATE) finish(n);
        if (TRAIN) {
            OT* p = (OT*)(a.ws + a.L.o_delta) + id * a.L.d;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                Slice<OT, 4> D;
                D.read(xs + ch * B::XT + B::XO, wv);
                D.write(p + (size_t)(NC * w.j + ch) * CH * 16, wv);
            }
        }
    }
    if (LATE && w.q.nt > 0) finish(w.q.nt - 1);
    if (TRAIN && w.q.nt > 0) store_state(w.q.nt - 1);
}

// Compute waves of the backward (as sc_fwd_walk). What does not depend on the state, Q^T (e^gam dO), is
// the side waves'.
template <class OT, int DK, int DV, int NC, bool SUM>
__device__ __forceinline__ void sc_bwd_walk(const ScArgs& a, const ScWalk& w, int wv, lds_char* b0, lds_char* b1,
                                            lds_char* xs) {
    using B = ScChainLds<OT, DK, NC, true>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NKB = B::NKB, F = B::F, NT = DK / 64;
    const int l = lane_id(), lq = l >> 4;
    const int nt = w.q.nt;
    ScState<OT, DK, NC, true> dS;
    dS.init(w, wv);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) dS.publish(xs, ch, wv);
    const size_t tstep = (size_t)a.Hv * a.L.t;
    const size_t id0 = ((size_t)(w.q.slot0 + max(nt - 1, 0)) * a.Hv + w.h) * a.L.t;
    const OT* tp = (const OT*)(a.ws + a.L.o_tt) + id0;
    const OT* mp = (const OT*)(a.ws + a.L.o_mt) + id0;
    ImgRows<OT, NS, true> T, M;  // rows of T^T and M^T, a step ahead
    if (nt > 0) {
        M.load(mp, wv);
        T.load(tp, wv);
    }
#pragma unroll 1
    for (int n = 0; n < nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vK{buf + B::K};
        sync_lds();  // A: the end-state gradient is published, the chunk's operands are in
        // dDelta = tail K dS' + M^T dO on this wave's tokens
        FT Kf[NKB];
        float e4[4], b4[4], t4[4];
        lds_get4<float>(buf + B::VEC + (SC_TAIL + 16 * wv + 4 * lq) * 4, t4);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            lds_char* xc = xs + ch * B::XT;
            const LPad<OT> vO{buf + B::V + ch * B::VT, 16};
            FT SB[NS][NKB], dO[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) dO[kb] = lfrag_colk8<OT>(vO, 0, 32 * kb);
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                if (ch == 0) Kf[kb] = lfrag_rowk8<OT>(vK, 16 * wv, 32 * kb);
#pragma unroll
                for (int p = 0; p < NS; ++p) SB[p][kb] = get_x<OT>(xc + B::XS + (p * NKB + kb) * F);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 Y[4], Z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[i] = Z[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p) mma(Z[2 * kb + p], M.f[p][kb], dO[kb]);
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p) mma(Y[2 * (kb & 1) + p], Kf[kb], SB[p][kb]);
            Y[0] = (Y[0] + Y[2]) + (Y[1] + Y[3]);
            Z[0] = (Z[0] + Z[2]) + (Z[1] + Z[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) Z[0][i] = (SUM && w.unit ? 0.f : Z[0][i]) + t4[i] * Y[0][i];
            put_split<OT>(xc + B::XX + (wv >> 1) * F, 2 * F, wv & 1, Z[0]);
        }
        lds_get4<float>(buf + B::VEC + (SC_E + 16 * wv + 4 * lq) * 4, e4);
        lds_get4<float>(buf + B::VEC + (SC_BETA + 16 * wv + 4 * lq) * 4, b4);
        const float ec = lds_load<float>(buf + B::VEC + SC_EC * 4);
        sync_lds();  // B: dDelta is published
        FT KT[NT][2];
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            lds_char* xc = xs + ch * B::XT;
            FT XB[NS][2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p) XB[p][kb] = get_x<OT>(xc + B::XX + (2 * p + kb) * F);
            if (ch == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) KT[t][kb] = lfrag_colk8<OT>(vK, 16 * (NT * wv + t), 32 * kb);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 D[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) D[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int p = 0; p < NS; ++p)
#pragma unroll
                    for (int r = 0; r < NS; ++r) mma(D[2 * p + r], T.f[r][kb], XB[p][kb]);
            D[0] = (D[0] + D[1]) + (D[2] + D[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) D[1][i] = -(b4[i] * e4[i]) * D[0][i];
            put_split<OT>(xc + B::XD + (wv >> 1) * F, 2 * F, wv & 1, D[1]);
            put_one<OT>(xc + B::XO + (wv >> 1) * F, wv & 1, D[0]);
        }
        sync_lds();  // C: dY is published, and the side waves' part of dS
        if (n + 1 < nt) {
            tp -= tstep;
            mp -= tstep;
        }
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            const lds_char* xc = xs + ch * B::XT;
            FT DB[NS][2];
            f32x4 P[NT];
#pragma unroll
            for (int p = 0; p < NS; ++p)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) DB[p][kb] = get_x<OT>(xc + B::XD + (2 * p + kb) * F);
#pragma unroll
            for (int t = 0; t < NT; ++t) P[t] = lds_load<f32x4>(xc + B::XP + ((NT * wv + t) * 64 + l) * 16);
            if (ch == 0) {
                M.load(mp, wv);
                T.load(tp, wv);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 s0 = dS.s[ch][t] * ec, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    mma(s0, KT[t][kb], DB[0][kb]);
                    if constexpr (NS == 2) mma(s1, KT[t][kb], DB[1][kb]);
                }
                dS.s[ch][t] = (s0 + s1) + P[t];
            }
            dS.publish(xs, ch, wv);
        }
    }
    dS.out(w, wv);
}

template <class OT, int DK, int DV, int NC, bool SUM>
__device__ __forceinline__ void sc_bwd_side(const ScArgs& a, const ScWalk& w, int wv, const lds_char* b0,
                                            const lds_char* b1, lds_char* xs) {
    using B = ScChainLds<OT, DK, NC, true>;
    using FT = typename Frag<OT>::type;
    constexpr int NS = B::NS, NT = DK / 64;
    const int l = lane_id(), lq = l >> 4;
    Slice<OT, DK / 16> S[NC];
    auto store_state = [&](int n) {  // the end-state gradient of walk index n
        OT* p = (OT*)(a.ws + a.L.o_ds) + ((size_t)(w.q.slot0 + (w.q.nt - 1 - n)) * a.Hv + w.h) * a.L.s;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) S[ch].write(p + (size_t)(NC * w.j + ch) * DK * 16, wv);
    };
#pragma unroll 1
    for (int n = 0; n < w.q.nt; ++n) {
        const lds_char* buf = (n & 1) ? b1 : b0;
        const LSwz<OT, DK> vQ{buf + B::Q};
        const size_t id = (size_t)(w.q.slot0 + (w.q.nt - 1 - n)) * a.Hv + w.h;
        sync_lds();  // A
        const bool give = !SUM || w.full;
        if (give && n > 0) store_state(n - 1);
        // Q^T (e^gam dO), rows: the keys of compute wave wv; one half of the tokens before B, the other after
        // it, so that neither barrier waits for these waves
        f32x4 P[NC][NT][2];
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
            for (int t = 0; t < NT; ++t) P[ch][t][0] = P[ch][t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto half = [&](int kb) {
            float s8[8];
            lds_get4<float>(buf + B::VEC + (SC_E + 32 * kb + 8 * lq) * 4, s8);
            lds_get4<float>(buf + B::VEC + (SC_E + 32 * kb + 8 * lq + 4) * 4, s8 + 4);
            FT qt[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) qt[t] = lfrag_colk8<OT>(vQ, 16 * (NT * wv + t), 32 * kb);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                const FT dO = lfrag_colk8<OT>(LPad<OT>{buf + B::V + ch * B::VT, 16}, 0, 32 * kb);
                FT hi, lo;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = s8[e] * to_f(dO[e]);
                    hi[e] = to_ot<OT>(x);
                    lo[e] = to_ot<OT>(x - to_f(hi[e]));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma(P[ch][t][0], qt[t], hi);
                    if constexpr (NS == 2) mma(P[ch][t][1], qt[t], lo);
                }
            }
        };
        half(0);
        sync_lds();  // B
        half(1);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                lds_store<f32x4>(xs + ch * B::XT + B::XP + ((NT * wv + t) * 64 + l) * 16,
                                 SUM && w.unit ? f32x4{0.f, 0.f, 0.f, 0.f} : P[ch][t][0] + P[ch][t][1]);
            if (give) S[ch].read(xs + ch * B::XT + B::XS, wv);
        }
        sync_lds();  // C
        if (!give) continue;
        OT* p = (OT*)(a.ws + a.L.o_dy) + id * a.L.d;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            Slice<OT, 4> Y;
            Y.read(xs + ch * B::XT + B::XO, wv);
            Y.write(p + (size_t)(NC * w.j + ch) * CH * 16, wv);
        }
    }
    if ((!SUM || w.full) && w.q.nt > 0) store_state(w.q.nt - 1);
}

// The sequence of rank r by length, the longest first (up to 64 packed sequences, one to a lane; more, and
// sequences of one length, are taken as they come): a long one started last would run on alone. Measured, 9
// sequences of 103 to 4000 tokens, 16 heads of 128: 115 us forward, 124 backward; as they come 144 and 156. What
// more than 64 lose by their order, forward, as they come and handed in longest first: 100 sequences of 20 to
// 2600 tokens, 4 heads of 128: 230 and 200 us, 16 heads 761 and 751; 300 sequences, 4 heads 595 and 545.
__device__ __forceinline__ int sc_ranked(const ScArgs& a, int r) {
    if (!a.cu || a.N > 64) return r;
    const int l = lane_id();
    const int len = l < a.N ? sc_seq(a.cu, a.T, l).len : -1;
    int rank = 0;
    for (int u = 0; u < a.N; ++u) {
        const int x = __builtin_amdgcn_readlane(len, u);
        rank += x > len || (x == len && u < l);
    }
    return __ffsll((unsigned long long)__ballot(l < a.N && rank == r)) - 1;
}

// Workgroup -> walk. Sequences of one length may be cut in a.nseg segments of a.seglen chunks (sc_segments),
// number i along the walk's direction. seg_e[.., i]: where segment i's walk ends; seg_p[.., i]: its transition,
// the end of a walk from the unit matrix. SUM: the walks that find those, of all segments but the last, each
// from zero (the first from the sequence's own start, and in full with a.lead), DV columns and for all but
// the first DK of the transition. Else: the segments themselves (with a.lead, all but the first), from the ends
// that k_sc_join has carried forward.
template <class OT, int DK, int DV, int NC, bool BWD, bool SUM>
__device__ __forceinline__ bool sc_walk_of(const ScArgs& a, const float* starts, float* ends, ScWalk& w) {
    constexpr int NJ = DV / (16 * NC), NJK = DK / (16 * NC);
    const int count = a.nseg - (SUM ? 1 : a.lead);
    int p, j;
    sc_chain_map(blockIdx.x, a.N * a.Hv * count, SUM ? NJ + NJK : NJ, !a.cu, p, j);
    const int i = p % count + (SUM ? 0 : a.lead), pair = p / count;
    w.h = pair % a.Hv;
    w.hk = w.h / a.R;
    const int s = sc_ranked(a, pair / a.Hv);
    w.q = sc_seq(a.cu, a.T, s);
    w.unit = SUM && j >= NJ;
    if (w.unit && i == 0) return false;
    w.full = !SUM || (i == 0 && a.lead);
    w.j = w.unit ? (j - NJ) % NJ : j;
    w.col = 16 * NC * (w.unit ? j - NJ : j);
    w.ld = w.unit ? DK : DV;
    const size_t st = (size_t)s * a.Hv + w.h, sg = st * a.nseg + i;
    float* const seg_e = (float*)(a.ws + a.L.o_seg);
    float* const seg_p = seg_e + (size_t)a.N * a.Hv * a.nseg * DK * DV;
    if (SUM) {
        w.start = i == 0 && starts ? starts + st * DK * DV : nullptr;
        w.end = w.unit ? seg_p + sg * DK * DK : seg_e + sg * DK * DV;
    } else {
        w.start = i > 0 ? seg_e + (sg - 1) * DK * DV : starts ? starts + st * DK * DV : nullptr;
        w.end = i + 1 == a.nseg && ends ? ends + st * DK * DV : nullptr;
    }
    if (a.nseg > 1) {
        const int c = a.seglen * (BWD ? a.nseg - 1 - i : i);  // its first chunk
        w.q.tok0 += 64LL * c;
        w.q.len = min(w.q.len - 64 * c, 64 * a.seglen);
        w.q.slot0 += c;
        w.q.nt = (w.q.len + 63) / 64;
    }
    return true;
}

constexpr int SC_THREADS = 64 * (2 * SC_NC + SC_NP);
static_assert(SC_THREADS == SC_CHAIN_THREADS, "as the host counts them");

template <class OT, int DK, int DV, int NC, bool TRAIN, bool OUT, bool SUM>
__global__ __launch_bounds__(SC_THREADS) void k_sc_fwd_chain(ScArgs a) {
    using B = ScChainLds<OT, DK, NC, false>;
    __shared__ __align__(16) char buf0[B::BYTES];
    __shared__ __align__(16) char buf1[B::BYTES];
    __shared__ __align__(16) char xch[B::XBYTES];
    __shared__ __align__(16) char pfslot[256];  // target of the prefetches, never read
    poison_lds((lds_char*)buf0, sizeof(buf0));
    poison_lds((lds_char*)buf1, sizeof(buf1));
    poison_lds((lds_char*)xch, sizeof(xch));
    poison_lds_done();
    ScWalk w;
    if (!sc_walk_of<OT, DK, DV, NC, false, SUM>(a, a.h0, a.ht, w)) return;
    const int wv = sc_wave();
    if (wv < SC_NC)
        sc_fwd_walk<OT, DK, DV, NC, SUM>(a, w, wv, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (wv < 2 * SC_NC)
        sc_fwd_side<OT, DK, DV, NC, TRAIN, OUT, SUM>(a, w, wv - SC_NC, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (w.q.nt > 0)
        sc_produce<OT, DK, DV, NC, false, OUT, SUM>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)pfslot, wv - 2 * SC_NC);
}

template <class OT, int DK, int DV, int NC, bool SUM>
__global__ __launch_bounds__(SC_THREADS) void k_sc_bwd_chain(ScArgs a) {
    using B = ScChainLds<OT, DK, NC, true>;
    __shared__ __align__(16) char buf0[B::BYTES];
    __shared__ __align__(16) char buf1[B::BYTES];
    __shared__ __align__(16) char xch[B::XBYTES];
    __shared__ __align__(16) char pfslot[256];  // target of the prefetches, never read
    poison_lds((lds_char*)buf0, sizeof(buf0));
    poison_lds((lds_char*)buf1, sizeof(buf1));
    poison_lds((lds_char*)xch, sizeof(xch));
    poison_lds_done();
    ScWalk w;
    if (!sc_walk_of<OT, DK, DV, NC, true, SUM>(a, a.dht, a.dh0, w)) return;
    const int wv = sc_wave();
    if (wv < SC_NC)
        sc_bwd_walk<OT, DK, DV, NC, SUM>(a, w, wv, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (wv < 2 * SC_NC)
        sc_bwd_side<OT, DK, DV, NC, SUM>(a, w, wv - SC_NC, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)xch);
    else if (w.q.nt > 0)
        sc_produce<OT, DK, DV, NC, true, true, SUM>(a, w, (lds_char*)buf0, (lds_char*)buf1, (lds_char*)pfslot, wv - 2 * SC_NC);
}

// Carries the segments' ends forward: E_i += P_i E_(i - 1) for i = 1 .. nseg - 2, so that E_i is where segment
// i + 1 starts. One workgroup of DK / 16 waves per (sequence, value head, 16 columns), wave w on rows
// 16 w .. + 15, E_(i - 1) in LDS. fp32 throughout, as the states are.
template <int DK, int DV>
__global__ __launch_bounds__(4 * DK) void k_sc_join(ScArgs a) {
    __shared__ __align__(16) float sE[DK * 17];
    poison_lds((lds_char*)sE, sizeof(sE));
    poison_lds_done();
    const int st = blockIdx.x / (DV / 16), col = 16 * (blockIdx.x % (DV / 16));
    const int l = lane_id(), li = l & 15, lq = l >> 4, r0 = 16 * sc_wave();
    float* const e0 = (float*)(a.ws + a.L.o_seg) + (size_t)st * a.nseg * DK * DV + col + li;
    const float* const p0 = (const float*)(a.ws + a.L.o_seg) + (size_t)a.N * a.Hv * a.nseg * DK * DV +
                            (size_t)st * a.nseg * DK * DK + (size_t)(r0 + li) * DK + 4 * lq;
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = e0[(size_t)(r0 + 4 * lq + i) * DV];
    for (int n = 1; n + 1 < a.nseg; ++n) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) sE[(r0 + 4 * lq + i) * 17 + li] = x[i];
        __syncthreads();
        float* e = e0 + (size_t)n * DK * DV;
        const float* p = p0 + (size_t)n * DK * DK;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = e[(size_t)(r0 + 4 * lq + i) * DV];
#pragma unroll
        for (int kb = 0; kb < DK / 16; ++kb) {
            const f32x4 pr = *(const f32x4*)(p + 16 * kb);
            const float a4[4] = {pr[0], pr[1], pr[2], pr[3]};
            float b4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b4[i] = sE[(16 * kb + 4 * lq + i) * 17 + li];
            mma_k16_f32(x, a4, b4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) e[(size_t)(r0 + 4 * lq + i) * DV] = x[i];
    }
}

// Column tiles a workgroup: with at most one 16-column walk for each compute unit, one; with two or more,
// walks queue, and two tiles to a workgroup share its operands, its barriers and their latencies (a step
// takes 1.4 times as long for twice the columns). Packed sequences may be uneven, which the host does not
// see, and then the longest walk, not their sum, sets the time: two tiles only from five walks a compute unit
// on, where they lose for neither kind. Measured, forward and training step in us, with two tiles and with one,
// 16 heads of 128, for sequences of 512 tokens and for log-uniform ones of 100 to 4000 with one of 4000:
//   2 walks a unit    38 and 44,   98 and 106      139 and  98,  346 and 255
//   4 walks a unit    59 and 71,  167 and 187      154 and 136,  441 and 402
//   4.5               81 and 87,  220 and 230      158 and 160,  491 and 479
//   5                 83 and 89,  228 and 237      187 and 223,  619 and 683
//   8                112 and 136, 330 and 381      259 and 305,  819 and 907
static hipError_t sc_column_tiles(const ScArgs& a, long long walks16, int& nc) {
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    nc = e == hipSuccess && walks16 >= (a.cu ? 5LL : 2LL) * cus ? 2 : 1;
    return e;
}

// The first segment and the others' ends, where there is more than one: summarise runs the SUM walks of nc
// column tiles.
template <int DK, int DV, class F>
static hipError_t sc_segment_ends(const ScArgs& a, hipStream_t stream, F summarise) {
    if (a.nseg <= 1) return hipSuccess;
    const long long tiles = (long long)a.N * a.Hv * (a.nseg - 1) * ((DV + DK) / 16);
    const int nc = tiles > 256 ? 2 : 1;
    summarise(nc, dim3((unsigned)(tiles / nc)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_sc_join<DK, DV>), dim3((unsigned)(a.N * a.Hv * (DV / 16))), dim3(4 * DK), 0, stream, a);
    return hipGetLastError();
}

template <class OT, int DK, int DV>
hipError_t launch_sc_fwd_chain_t(const ScArgs& a, bool train, hipStream_t stream) {
    int nc;
    const long long walks = (long long)a.N * a.Hv * (a.nseg - a.lead) * (DV / 16);
    hipError_t e = sc_column_tiles(a, walks, nc);
    if (e != hipSuccess) return e;
    auto pick2 = [&](auto n, auto sum) {
        constexpr int NC = decltype(n)::value;
        constexpr bool SUM = decltype(sum)::value;
        return !train ? k_sc_fwd_chain<OT, DK, DV, NC, false, true, SUM>
               : a.o  ? k_sc_fwd_chain<OT, DK, DV, NC, true, true, SUM> : k_sc_fwd_chain<OT, DK, DV, NC, true, false, SUM>;
    };
    auto pick = [&](int n, auto sum) {
        return n == 2 ? pick2(std::integral_constant<int, 2>{}, sum) : pick2(std::integral_constant<int, 1>{}, sum);
    };
    e = sc_segment_ends<DK, DV>(a, stream, [&](int n, dim3 grid) {
        hipLaunchKernelGGL(pick(n, std::true_type{}), grid, dim3(SC_THREADS), 0, stream, a);
    });
    if (e != hipSuccess) return e;
    auto k = pick(nc, std::false_type{});
    hipLaunchKernelGGL(k, dim3((unsigned)(walks / nc)), dim3(SC_THREADS), 0, stream, a);
    return hipGetLastError();
}
template <class OT, int DK, int DV>
hipError_t launch_sc_bwd_chain_t(const ScArgs& a, hipStream_t stream) {
    int nc;
    const long long walks = (long long)a.N * a.Hv * (a.nseg - a.lead) * (DV / 16);
    hipError_t e = sc_column_tiles(a, walks, nc);
    if (e != hipSuccess) return e;
    e = sc_segment_ends<DK, DV>(a, stream, [&](int n, dim3 grid) {
        auto k = n == 2 ? k_sc_bwd_chain<OT, DK, DV, 2, true> : k_sc_bwd_chain<OT, DK, DV, 1, true>;
        hipLaunchKernelGGL(k, grid, dim3(SC_THREADS), 0, stream, a);
    });
    if (e != hipSuccess) return e;
    auto k = nc == 2 ? k_sc_bwd_chain<OT, DK, DV, 2, false> : k_sc_bwd_chain<OT, DK, DV, 1, false>;
    hipLaunchKernelGGL(k, dim3((unsigned)(walks / nc)), dim3(SC_THREADS), 0, stream, a);
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
