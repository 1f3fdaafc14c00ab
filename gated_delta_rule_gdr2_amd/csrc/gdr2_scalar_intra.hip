// Gated delta rule with scalar gates: the kernels that are parallel over chunks (see
// gdr2_scalar.hpp for the equations). Forward: T = (I + A)^-1 and M of every chunk and value
// head. Backward: the gradients, from the states and their gradients that the chains left.
#include "gdr2_intra_common.hpp"
#include "gdr2_scalar_device.hpp"

namespace gdr2 {

// A log-decay as it enters the running sum: e^-256 is zero in 32 bits (the smallest number there is e^-103),
// so a stronger one says no more, and every decay across the token, gradients included, is the same exact
// zero. Left as it is, -1e18 would take the digits of all later sums of its chunk, and two of the type's
// lowest value would pass the range in which gam is kept (both gave wrong results and NaN). Each at -256 at
// least, gam stays above -2^14. NaN passes through.
__device__ __forceinline__ double log_decay(float g) { return g < -256.f ? -256.0 : (double)g; }

// gam = running sum of g over the chunk's rows (lane = row), in 64 bits: the decays are exponentials
// of differences of gam, and in 32 bits a strong decay early in the chunk (gam of some thousands)
// would cost a later weak one its digits.
__device__ __forceinline__ double wave_scan(double x) {
    const int l = lane_id();
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(x, o);
        if (l >= o) x += y;
    }
    return x;
}

// upper 16x16 block (R, I), I > R, number u = 0..5
__device__ __forceinline__ void sc_upper_ri(int u, int& R, int& I) {
    R = u < 3 ? 0 : (u < 5 ? 1 : 2);
    I = u < 3 ? u + 1 : (u < 5 ? u - 1 : 3);
}

// x + the value N lanes up in the row of 16 (zero past its end)
template <int N>
__device__ __forceinline__ float row_suffix_step(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x100 + N, 0xF, 0xF, false));
}
// sum over 8 neighbouring lanes (of those that share l / 8), in the first of them
__device__ __forceinline__ float row_sum8(float x) {
    x = row_suffix_step<1>(x);
    x = row_suffix_step<2>(x);
    return row_suffix_step<4>(x);
}

// D_ri = exp(gam_r - gam_i) from gam held as a float and its remainder
template <class OT>
__device__ __forceinline__ float decay(float rhi, float rlo, float ihi, float ilo) {
    return exp_op<OT>((rhi - ihi) + (rlo - ilo));
}

// Inverse T of the unit lower-triangular I + A (A and T fp32 in LDS, 4 waves; the upper blocks of T
// are zero already). Wave w solves diagonal block w by forward substitution, lane li for column li
// (substitution, not a product of powers of A: those grow like binomials when keys repeat); then
// T_RI = -T_RR sum_{K = I}^{R - 1} A_RK T_KI on fp32 MFMA, one level of blocks at a time.
__device__ __forceinline__ void sc_inverse(const lds_char* sA, lds_char* sT) {
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Lane ln = fresh_lane();
    const int li = ln.li, lq = ln.lq;
    auto A = [&](int r, int c) { return sA + swz<float, CH>(r, c) * 4; };
    auto Tp = [&](int r, int c) { return sT + swz<float, CH>(r, c) * 4; };
    {
        // row r of the block: its chunk i4 / 4 sits at (4 wv + i4 / 4) ^ f(r), f(r) known here
        const lds_char* base[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) base[j] = sA + 16 * wv * CH * 4 + ((4 * wv) ^ (4 * j)) * 16;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int f = swz_f<float, CH>(r);
            float acc = r == li ? 1.f : 0.f;
#pragma unroll
            for (int i4 = 0; i4 < r; i4 += 4) {
                const f32x4 row = lds_load<f32x4>(base[f >> 2] + r * CH * 4 + ((i4 / 4) ^ (f & 3)) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i4 + i < r) acc -= row[i] * x[i4 + i];
            }
            x[r] = acc;
        }
        if (lq == 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) lds_store<float>(Tp(16 * wv + r, 16 * wv + li), x[r]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int lev = 1; lev < NBLK; ++lev) {
        if (wv < NBLK - lev) {
            const int I = wv, R = wv + lev;
            f32x4 z = {0.f, 0.f, 0.f, 0.f}, t = z;
#pragma unroll
            for (int k = 0; k < lev; ++k) {
                float a4[4], b4[4];
                lds_get4<float>(A(16 * R + li, 16 * (I + k) + 4 * lq), a4);
#pragma unroll
                for (int e = 0; e < 4; ++e) b4[e] = lds_load<float>(Tp(16 * (I + k) + 4 * lq + e, 16 * I + li));
                mma_k16_f32(z, a4, b4);
            }
            float a4[4];
            const float b4[4] = {z[0], z[1], z[2], z[3]};
            lds_get4<float>(Tp(16 * R + li, 16 * R + 4 * lq), a4);
            mma_k16_f32(t, a4, b4);
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_store<float>(Tp(16 * R + 4 * lq + i, 16 * I + li), -t[i]);
        }
        __syncthreads();
    }
}

// four elements and their remainders to a pair of images
template <class OT>
__device__ __forceinline__ void put_parts(OT* p, const f32x4& x) {
    if constexpr (sizeof(OT) == 2) {
        bf16x4 hi, lo;
        split4(x, hi, lo);
        *(bf16x4*)p = hi;
        *(bf16x4*)(p + CH * CH) = lo;
    } else {
        *(f32x4*)p = x;
    }
}

// One workgroup of four waves per (chunk slot, value head): k k^T and q k^T on the raw rows, then A, its
// inverse and M with the head's decay and beta. (One workgroup per key head, which would form the
// products once for all of its value heads, was no faster where many run, 36 and 35 us for 2 x 4096 tokens
// and 16 heads before T^T and M^T were written, and slower where few do, 15.7 and 10 us for three chunks
// in fp32.)
// Bound by HBM traffic in the large: reads q and k, writes T, M and the row factors, for training T^T and
// M^T too, 52 (training 76) KB a chunk and value head at d_k = 128 with Hk = Hv; 51 us for 16384 tokens and
// 16 heads, 38 us for 2 x 4096 in training, 4.1 TB/s both. In the small by latencies one behind the other, the
// tiles' copies, the products, the gates (loaded and scanned in 64 bits by one wave while three wait) and the
// blocked inverse: 11.5 us for three chunks.
template <class OT, int DK, bool TRAIN>
__global__ __launch_bounds__(256, 4) void k_sc_prep(ScArgs a) {
    constexpr int KB = DK / 32, ES = sizeof(OT);
    constexpr int TILE = CH * DK * ES, SQ = CH * CH * 4;
    constexpr int BUF = 2 * TILE > 2 * SQ ? 2 * TILE : 2 * SQ;
    __shared__ __align__(16) char smem_[BUF];
    __shared__ __align__(16) char svec_[SC_VEC * 4];
    lds_char* smem = (lds_char*)smem_;
    lds_char* sV = (lds_char*)svec_;
    poison_lds(smem, sizeof(smem_));
    poison_lds(sV, sizeof(svec_));
    poison_lds_done();
    const int tid = threadIdx.x, l = tid & 63, li = l & 15, lq = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / a.R;
    if (a.cu && a.zero_rest && a.o) zero_rest_rows<OT>(a, slot, a.o, a.Hv, h, 1, a.DV);
    ScSeq q;
    int c;
    if (!sc_slot(a.cu, a.T, a.N, slot, q, c)) return;
    const long long row0 = q.tok0 + 64LL * c;
    const int nvalid = min(CH, q.len - CH * c);
    const size_t rsk = (size_t)a.Hk * DK;
    lds_char* sK = smem;
    lds_char* sQ = smem + TILE;
    dma_rows<OT, DK, 4>((const OT*)a.k + row0 * rsk + (size_t)hk * DK, rsk, nvalid, sK, wv);
    dma_rows<OT, DK, 4>((const OT*)a.q + row0 * rsk + (size_t)hk * DK, rsk, nvalid, sQ, wv);
    zero_tail_rows<OT, DK, 256>(sK, nvalid);
    zero_tail_rows<OT, DK, 256>(sQ, nvalid);
    wait_vm<0>();
    __syncthreads();
    // block pairs p = wv, wv + 4, wv + 8 of the lower triangle, as transposed tiles: lane (li, lq)
    // holds rows 16 R + li, columns 16 I + 4 lq + i
    const LSwz<OT, DK> vK{sK}, vQ{sQ};
    f32x4 kk[3], qk[3], kq[3];  // kq: training, the tile of q k^T itself (rows 16 R + 4 lq + i, columns 16 I + li)
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int p = wv + 4 * n;
        kk[n] = qk[n] = kq[n] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (p < NPAIR) {
            int R, I;
            pair_ri(p, R, I);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const auto fi = lfrag_rowk8<OT>(vK, 16 * I, 32 * kb);
                mma(kk[n], fi, lfrag_rowk8<OT>(vK, 16 * R, 32 * kb));
                const auto fq = lfrag_rowk8<OT>(vQ, 16 * R, 32 * kb);
                mma(qk[n], fi, fq);
                if (TRAIN) mma(kq[n], fq, fi);
            }
        }
    }
    __syncthreads();  // the tiles are dead: A and T take their place
    lds_char* sA = smem;
    lds_char* sT = smem + SQ;
    for (int idx = tid; idx < 6 * 64; idx += 256) {  // the upper blocks of T stay zero
        int R, I;
        sc_upper_ri(idx / 64, R, I);
        const int e = idx % 64;
        lds_store<f32x4>(sT + swz<float, CH>(16 * R + e / 4, 16 * I + 4 * (e % 4)) * 4, f32x4{});
    }
    const size_t id = (size_t)slot * a.Hv + h;
    if (wv == 0) {
        const bool ok = l < nvalid;
        const size_t at = (size_t)(row0 + l) * a.Hv + h;
        const double gam = wave_scan(ok ? log_decay(to_f(((const OT*)a.g)[at])) : 0.0);
        const double gc = __shfl(gam, 63);
        const float hi = (float)gam, lo = (float)(gam - (double)hi);
        const float v[6] = {ok ? exp_op<OT>(hi) * (1.f + lo) : 0.f, ok ? to_f(((const OT*)a.beta)[at]) : 0.f,
                            ok ? exp_op<OT>((float)(gc - gam)) : 0.f, hi, lo, exp_op<OT>((float)gc)};
        float* vec = (float*)(a.ws + a.L.o_vec) + id * a.L.vec;
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            lds_store<float>(sV + (64 * i + l) * 4, v[i]);
            vec[64 * i + l] = v[i];
        }
    }
    __syncthreads();
    OT* m = (OT*)(a.ws + a.L.o_m) + id * a.L.m;
    OT* mt = (OT*)(a.ws + a.L.o_mt) + id * a.L.t;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int p = wv + 4 * n;
        if (p < NPAIR) {
            int R, I;
            pair_ri(p, R, I);
            const int r = 16 * R + li, i0 = 16 * I + 4 * lq;
            const float rhi = lds_load<float>(sV + (SC_GHI + r) * 4), rlo = lds_load<float>(sV + (SC_GLO + r) * 4);
            const float beta = lds_load<float>(sV + (SC_BETA + r) * 4);
            float ihi[4], ilo[4], av[4];
            lds_get4<float>(sV + (SC_GHI + i0) * 4, ihi);
            lds_get4<float>(sV + (SC_GLO + i0) * 4, ilo);
            f32x4 mv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // above the diagonal the exponent would be positive: there the product is dropped
                const float d = i0 + i <= r ? decay<OT>(rhi, rlo, ihi[i], ilo[i]) : 0.f;
                mv[i] = d == 0.f ? 0.f : d * qk[n][i];
                av[i] = i0 + i < r && d != 0.f ? beta * d * kk[n][i] : 0.f;
            }
            f32x4 a4 = {av[0], av[1], av[2], av[3]};
            lds_store<f32x4>(sA + swz<float, CH>(r, i0) * 4, a4);
            const float mv4[4] = {mv[0], mv[1], mv[2], mv[3]};
            st4(m + fimg<OT, CH>(r, i0), mv4);
            if (TRAIN) {  // M^T: row 16 I + li, columns 16 R + 4 lq ..
                const int ti = 16 * I + li, r0 = 16 * R + 4 * lq;
                const float chi = lds_load<float>(sV + (SC_GHI + ti) * 4), clo = lds_load<float>(sV + (SC_GLO + ti) * 4);
                float qhi[4], qlo[4];
                lds_get4<float>(sV + (SC_GHI + r0) * 4, qhi);
                lds_get4<float>(sV + (SC_GLO + r0) * 4, qlo);
                f32x4 x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = ti <= r0 + i ? decay<OT>(qhi[i], qlo[i], chi, clo) : 0.f;
                    x[i] = d == 0.f ? 0.f : d * kq[n][i];
                }
                put_parts<OT>(mt + fimg<OT, CH>(ti, r0), x);
            }
        }
    }
    if (wv < 2) {  // the two zero blocks in the fragments that are read (sc_img_zero)
        const int R = 2 * wv, I = R + 1;
        const float z[4] = {0.f, 0.f, 0.f, 0.f};
        st4(m + fimg<OT, CH>(16 * R + li, 16 * I + 4 * lq), z);
        if (TRAIN) put_parts<OT>(mt + fimg<OT, CH>(16 * I + li, 16 * R + 4 * lq), f32x4{0.f, 0.f, 0.f, 0.f});
    }
    __syncthreads();
    sc_inverse(sA, sT);
    // T out (and for training T^T), 4 columns of a row at a time
    OT* t = (OT*)(a.ws + a.L.o_t) + id * a.L.t;
    OT* tt = (OT*)(a.ws + a.L.o_tt) + id * a.L.t;
#pragma unroll
    for (int i = 0; i < CH * CH / 4 / 256; ++i) {
        const int idx = tid + 256 * i, r = idx / 16, c0 = 4 * (idx % 16);
        if (!sc_img_zero<false>(i, c0 / 32))
            put_parts<OT>(t + fimg<OT, CH>(r, c0), lds_load<f32x4>(sT + swz<float, CH>(r, c0) * 4));
        if (TRAIN) {
            // lanes on 16 neighbouring columns of four rows: row c of T^T, columns r0 ..
            const int ct = 16 * (idx / 64 % 4) + idx % 16, r0 = 16 * (idx / 256) + 4 * (idx / 16 % 4);
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = lds_load<float>(sT + swz<float, CH>(r0 + e, ct) * 4);
            if (!sc_img_zero<true>(ct / 16, r0 / 32)) put_parts<OT>(tt + fimg<OT, CH>(ct, r0), x);
        }
    }
}

// ============================================================================ gradients
template <class OT, int DK, int DV, bool MULTI>
struct ScGradLds {
    static constexpr int ES = sizeof(OT), NS = Split<OT>::NS;
    static constexpr int NW = 8;               // waves
    static constexpr int KW = DK / 16;         // 16-row tiles of key channels, one a wave;
    static constexpr int TPW = 4 * KW / NW;    // token tiles of a wave: all four, or half of them where KW = 4
    static constexpr int SQ = CH * CH * ES;
    static constexpr int TK = CH * DK * ES, TV = CH * DV * ES;
    static constexpr int K = 0;             // raw k rows, swizzled
    static constexpr int Q = K + TK;        // raw q rows: MULTI
    static constexpr int HEAD = MULTI ? Q + TK : Q;  // a head's region (MULTI: two of them). In it:
    static constexpr int DO = 0;            // dO rows, swizzled
    static constexpr int DEL = DO + TV;     // Delta, dY: slices [DV / 16][64][16]
    static constexpr int DY = DEL + TV;
    static constexpr int P = DO;            // after the pair products: P, R / beta, R, P's second part [64][64]
    static constexpr int RP = P + SQ;
    static constexpr int R = RP + SQ;
    static constexpr int PL = R + SQ;       // (bf16)
    static constexpr int QL = PL + (NS == 2 ? SQ : 0);  // and raw q rows: one head
    static constexpr int ODQ = DO;          // at the end: dq and dk rows on their way out
    static constexpr int ODK = ODQ + TK;
    static constexpr int AFTER = MULTI ? QL : QL + TK;
    static constexpr int MX = 3 * TV > AFTER ? 3 * TV : AFTER;
    static constexpr int VEC = MX > 2 * TK ? MX : 2 * TK;  // the row factors (copied by two waves, 1 KB each)
    static constexpr int REGION = VEC + 2048;
    static_assert(SC_VEC * 4 > 1024 && SC_VEC * 4 <= 2048, "the row factors are two waves' copies");
    static constexpr int ROWP = HEAD + (MULTI ? 2 : 1) * REGION;  // per block pair: row and column sums of N
    static constexpr int COLP = ROWP + NPAIR * 16 * 4;
    static constexpr int DOTS = COLP + NPAIR * 16 * 4;  // per key tile and row: q.dq_s, k.dx_s, k.dk_s, k.G
    static constexpr int DOTV = DOTS + 4 * KW * CH * 4; // per row: dY.Delta / beta, or dY.v
    static constexpr int SS = DOTV + CH * 4;            // per key tile: <dS', S>
    static constexpr int RED = SS + KW * 4;             // 6 sums a row
    static constexpr int BYTES = RED + 6 * CH * 4;
};

// 64 raw rows into a swizzled tile, rows from nvalid on repeating the last (they meet zeros only)
template <class OT, int RL, int NW>
__device__ __forceinline__ void dma_rows_clamped(const OT* base, size_t rs, int nvalid, lds_char* tile, int wv) {
    constexpr int EPC = 16 / (int)sizeof(OT), NCH = RL / EPC, RPI = 64 / NCH, NI = CH / RPI;
    const int l = lane_id();
#pragma unroll
    for (int n = 0; n < NI; n += NW) {
        const int row = (n + wv) * RPI + l / NCH, c = (l % NCH) ^ swz_f<OT, RL>(row);
        const char* src = (const char*)(base + (size_t)min(row, nvalid - 1) * rs + c * EPC);
        __builtin_amdgcn_global_load_lds(src, (lds_void*)(tile + (n + wv) * 1024), 16, 0, 0);
    }
}

// dbeta = dY.(v - k^T X) with X the state before the token, decayed, and beta (v - k^T X) is Delta. The other
// form, dY.v + k.G, is a difference of terms of the size of v: where the state already predicts v, as a trained
// one does, the bf16 roundings of S and of the intermediates in G would stay at that size (normwise errors in
// bf16 where v - k^T X is a tenth and a thirtieth of v: 1.2e-2 and 3.9e-2 against 2.9e-3). It is left for a
// beta so small that Delta, a product with it, would leave the normal numbers.
__device__ __forceinline__ bool sc_dbeta_by_delta(float beta) { return fabsf(beta) >= 0x1p-32f; }

// One workgroup of eight waves per (chunk slot, key head), each wave a 16-row tile of key channels
// (two waves to a tile, half the tokens each, where d_k = 64): the gradients of the
// group's value heads one after another, dq and dk summed over them in fp32 registers (value heads
// that share a key head need no second pass and no atomics). Per value head
//   dq_s = e^gam S dO, dx_s = -e^gam S dY, dk_s = tail dS' Delta   (columns of S, dS': fragments
//     straight from the workspace; dO, dY, Delta from LDS, which every wave reads whole)
//   dM = lower(dO Delta^T), dA = -strict(dY Delta^T), q k^T, k k^T in 16x16 block pairs, from which
//   P = D dM, R = beta D dA and N = P q.k + R k.k, the derivative of every D_ri times D_ri
//   dq = dq_s + P K,  G = dx_s + (R / beta) K,  dk = P^T Q + R^T K + beta G + dk_s
//   dv = beta dY,  dbeta = dY.Delta / beta, or dY.v + k.G where beta is next to nothing (sc_dbeta_by_delta)
//   dg_t = sum_{r >= t} (row_r - col_r of N + q.dq_s + beta k.dx_s) + sum_{i < t} k.dk_s + e^gamC <dS', S>
// In bf16 P enters the last products in two parts, a value and what its rounding left over: dq and dk are off by
// 2.4e-3 (2.9e-3 with one, and 329 us instead of 330 for the whole step of 2 x 4096 tokens, 407 instead of 411
// for the packed one), of which 1.7e-3 are their own rounding. R and R / beta take one part, the smaller terms
// beside what the saved arrays' roundings leave. N and all sums stay in 32 bits.
// The last line sums only terms that carry the decay across t: the diagonal of N, which does not
// depend on the decay, is left out, so that a strong decay leaves a small dg and no cancellation.
//
// A chunk and head moves 208 KB (d = 128, bf16), which at the rate of HBM is two thirds of the time.
// One value head a key head: two workgroups a compute unit, one loading while the other works, which
// is what the LDS layout (q enters LDS only when dO, Delta and dY have left it) and the register bound
// are for. MULTI, more than one: around a loop over heads the registers are not enough for two workgroups
// (84 spilled), so one has the compute unit, keeps q in LDS and loads the next head while this one is
// worked on. Measured, d = 128, bf16: 100 us at 2 x 4096 tokens, 16 heads (4.4 TB/s); 135 us at 8859 packed
// tokens, 8 key heads with 2 value heads each (3.0 TB/s, five rounds of workgroups of which the last is half
// empty; without the loads ahead 144 us).
template <class OT, int DK, int DV, bool MULTI>
__global__ __launch_bounds__(512, sizeof(OT) == 2 && !MULTI ? 4 : 2) void k_sc_grad(ScArgs a) {
    using LS = ScGradLds<OT, DK, DV, MULTI>;
    using FT = typename Frag<OT>::type;
    constexpr int ES = sizeof(OT), NW = LS::NW, KW = LS::KW, TPW = LS::TPW, NTHR = 64 * NW, KB = DK / 32, VB = DV / 32;
    constexpr int PPW = (NPAIR + NW - 1) / NW;  // block pairs of a wave
    extern __shared__ __align__(16) char smem_[];
    lds_char* sm = (lds_char*)smem_;
    poison_lds(sm, LS::BYTES);
    poison_lds_done();
    const int slot = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk;
    if (a.cu && a.zero_rest) {
        zero_rest_rows<OT>(a, slot, a.dq, a.Hk, hk, 1, DK);
        zero_rest_rows<OT>(a, slot, a.dk, a.Hk, hk, 1, DK);
        zero_rest_rows<OT>(a, slot, a.dv, a.Hv, hk * a.R, a.R, DV);
        zero_rest_rows<OT>(a, slot, a.dg, a.Hv, hk * a.R, a.R, 1);
        zero_rest_rows<OT>(a, slot, a.dbeta, a.Hv, hk * a.R, a.R, 1);
    }
    ScSeq q;
    int c;
    if (!sc_slot(a.cu, a.T, a.N, slot, q, c)) return;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long row0 = q.tok0 + 64LL * c;
    const int nvalid = min(CH, q.len - CH * c);
    const size_t rsk = (size_t)a.Hk * DK, rsv = (size_t)a.Hv * DV;
    const size_t k0 = row0 * rsk + (size_t)hk * DK;
    const LSwz<OT, DK> vK{sm + LS::K};
    dma_rows_clamped<OT, DK, NW>((const OT*)a.k + k0, rsk, nvalid, sm + LS::K, wv);
    if (MULTI) dma_rows_clamped<OT, DK, NW>((const OT*)a.q + k0, rsk, nvalid, sm + LS::Q, wv);
    const int kw = wv % KW, t0 = TPW * (wv / KW);  // this wave's key tile and first token tile
    f32x4 dq[TPW], dk[TPW];  // transposed tiles: keys 16 kw + 4 lq + i, tokens 16 (t0 + t) + li
#pragma unroll
    for (int t = 0; t < TPW; ++t) dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    // What a value head brings: dO, Delta, dY and the row factors to LDS; this wave's key rows of S and dS'
    // (K = value column) and v (16 bytes of a row a lane, rows past the end zero) to registers
    constexpr int EPC = 16 / ES, LPR = DV / EPC, NVL = CH * LPR / NTHR;
    typedef OT VT __attribute__((ext_vector_type(EPC)));
    FT fS[VB], fdS[VB];
    VT gv[NVL];
    auto load_lds = [&](int h, lds_char* hd) {
        const size_t id = (size_t)slot * a.Hv + h;
        const int l = lane_id();
        dma_rows<OT, DV, NW>((const OT*)a.dout + row0 * rsv + (size_t)h * DV, rsv, nvalid, hd + LS::DO, wv);
        zero_tail_rows<OT, DV, NTHR>(hd + LS::DO, nvalid);
        const char* gDel = a.ws + a.L.o_delta + id * a.L.d * ES;
        const char* gDy = a.ws + a.L.o_dy + id * a.L.d * ES;
#pragma unroll
        for (int n = 0; n < LS::TV / 1024; n += NW) {
            const int kb = (n + wv) * 1024;
            __builtin_amdgcn_global_load_lds(gDel + kb + l * 16, (lds_void*)(hd + LS::DEL + kb), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(gDy + kb + l * 16, (lds_void*)(hd + LS::DY + kb), 16, 0, 0);
        }
        if (wv < 2) {  // (the second wave's upper lanes: again what its lower lanes copy)
            const int piece = wv == 0 ? l : 64 + l % ((SC_VEC * 4 - 1024) / 16);
            const char* src = a.ws + a.L.o_vec + id * a.L.vec * 4 + piece * 16;
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(hd + LS::VEC + wv * 1024), 16, 0, 0);
        }
    };
    auto load_s = [&](int h) {
        const size_t id = (size_t)slot * a.Hv + h;
#pragma unroll
        for (int kb = 0; kb < VB; ++kb) {
            fS[kb] = gfrag_slice<OT, DK>((const OT*)(a.ws + a.L.o_s) + id * a.L.s, 16 * kw, kb);
            fdS[kb] = gfrag_slice<OT, DK>((const OT*)(a.ws + a.L.o_ds) + id * a.L.s, 16 * kw, kb);
        }
    };
    auto load_v = [&](int h) {
#pragma unroll
        for (int i = 0; i < NVL; ++i) {
            const int u = threadIdx.x + NTHR * i, rr = u / LPR;
            const OT* p = (const OT*)a.v + (row0 + rr) * rsv + (size_t)h * DV + EPC * (u % LPR);
            gv[i] = rr < nvalid ? *(const VT*)p : VT{};
        }
    };
    load_lds(hk * a.R, sm + LS::HEAD);
    load_s(hk * a.R);
    load_v(hk * a.R);

#pragma unroll 1
    for (int hh = 0; hh < (MULTI ? a.R : 1); ++hh) {
        const int h = hk * a.R + hh;
        const size_t v0 = row0 * rsv + (size_t)h * DV;
        lds_char* hd = sm + LS::HEAD + (MULTI ? (hh & 1) * LS::REGION : 0);
        const LSwz<OT, DK> vQ{MULTI ? sm + LS::Q : hd + LS::QL};
        const LSwz<OT, DV> vO{hd + LS::DO};
        const LSlice<OT, CH> vDel{hd + LS::DEL}, vDy{hd + LS::DY};
        const LSwz<OT, CH> vP{hd + LS::P}, vPl{hd + LS::PL}, vRp{hd + LS::RP}, vR{hd + LS::R};
        Lane ln = fresh_lane();
        const int li = ln.li, lq = ln.lq, l = li + 16 * lq, tid = 64 * wv + l;
        const bool more = MULTI && hh + 1 < a.R;
        typename Raw4<OT>::type qv[TPW];  // q of this wave's tokens and keys
        if (!MULTI) {
#pragma unroll
            for (int t = 0; t < TPW; ++t)
                qv[t] = *(const typename Raw4<OT>::type*)(
                    (const OT*)a.q + k0 + (size_t)min(16 * (t0 + t) + li, nvalid - 1) * rsk + 16 * kw + 4 * lq);
        }
        wait_vm<0>();
        sync_lds();  // this head is in LDS, and the head before is done with its region
        if (more) load_lds(h + 1, sm + LS::HEAD + ((hh + 1) & 1) * LS::REGION);

        // ---- the states' parts
        auto dot4 = [&](const float (&y)[4], const f32x4& x, int t, int which) {
            // sum over this wave's keys of y x, tokens 16 (t0 + t) + li
            const float s = sum_lq((y[0] * x[0] + y[1] * x[1]) + (y[2] * x[2] + y[3] * x[3]));
            if (lq == 0) lds_store<float>(sm + LS::DOTS + ((which * KW + kw) * CH + 16 * (t0 + t) + li) * 4, s);
        };
        f32x4 G[TPW];
        ln = fresh_lane();
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            const int tt = t0 + t;
            f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x, z = x;
#pragma unroll
            for (int kb = 0; kb < VB; ++kb) {
                mma(x, fS[kb], frag_rows<OT>(ln, vO, 16 * tt, 32 * kb));
                mma(y, fS[kb], frag_rows<OT>(ln, vDy, 16 * tt, 32 * kb));
                mma(z, fdS[kb], frag_rows<OT>(ln, vDel, 16 * tt, 32 * kb));
            }
            x = x * lds_load<float>(hd + LS::VEC + (SC_E + 16 * tt + ln.li) * 4);
            G[t] = y * -lds_load<float>(hd + LS::VEC + (SC_E + 16 * tt + ln.li) * 4);
            z = z * lds_load<float>(hd + LS::VEC + (SC_TAIL + 16 * tt + ln.li) * 4);
            dq[t] += x;
            dk[t] += z;
            float kx[4];
            float qx[4];
            if (MULTI) {
                lds_get4<OT>(vQ.p + vQ.off(16 * tt + ln.li, 16 * kw + 4 * ln.lq), qx);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) qx[i] = to_f(qv[t][i]);
            }
            lds_get4<OT>(vK.p + vK.off(16 * tt + ln.li, 16 * kw + 4 * ln.lq), kx);
            dot4(qx, x, t, 0);
            dot4(kx, G[t], t, 1);
            dot4(kx, z, t, 2);
            __builtin_amdgcn_sched_barrier(0);
        }
        {
            float s = 0.f;
#pragma unroll
            for (int kb = 0; kb < VB; ++kb)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += to_f(fS[kb][i]) * to_f(fdS[kb][i]);
            s = row_sum16(s);
            s = (lane_value(s, 0) + lane_value(s, 16)) + (lane_value(s, 32) + lane_value(s, 48));
            if (l == 0) lds_store<float>(sm + LS::SS + kw * 4, s);  // (the same from both waves of a key tile)
        }
        if (more) {
            __builtin_amdgcn_sched_barrier(0);
            load_s(h + 1);
        }

        // ---- dv = beta dY and the row's part of dbeta, 16 bytes of a row a lane
#pragma unroll
        for (int i = 0; i < NVL; ++i) {
            const int u = tid + NTHR * i, rr = u / LPR, col = EPC * (u % LPR);
            const VT y = lds_load<VT>(vDy.p + vDy.off(rr, col));
            const VT del = lds_load<VT>(vDel.p + vDel.off(rr, col));
            const float b = lds_load<float>(hd + LS::VEC + (SC_BETA + rr) * 4);
            const bool by_delta = sc_dbeta_by_delta(b);
            float s = 0.f;
            VT d;
#pragma unroll
            for (int j = 0; j < EPC; ++j) {
                s += to_f(y[j]) * to_f(by_delta ? del[j] : gv[i][j]);
                d[j] = to_ot<OT>(b * to_f(y[j]));
            }
            if (rr < nvalid) *(VT*)((OT*)a.dv + v0 + rr * rsv + col) = d;
            s = LPR == 16 ? row_sum16(s) : row_sum8(s);
            if (u % LPR == 0) lds_store<float>(sm + LS::DOTV + rr * 4, by_delta ? s / b : s);
        }
        if (more) load_v(h + 1);
        __builtin_amdgcn_sched_barrier(0);

        // ---- block pairs (rows 16 R + li, columns 16 I + 4 lq + i)
        f32x4 fP[PPW], fRp[PPW];
        ln = fresh_lane();
#pragma unroll
        for (int n = 0; n < PPW; ++n) {
            const int p = wv + NW * n;
            if (p < NPAIR) {
                int R, I;
                pair_ri(p, R, I);
                const int r = 16 * R + ln.li, i0 = 16 * I + 4 * ln.lq;
                // one head: the rows of q come from memory (this chunk's are in cache by now)
                FT fq[KB];
                const OT* qp = (const OT*)a.q + k0 + (size_t)min(r, nvalid - 1) * rsk + 8 * ln.lq;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    if constexpr (MULTI) {
                        fq[kb] = frag_rows<OT>(ln, vQ, 16 * R, 32 * kb);
                    } else if constexpr (ES == 2) {
                        fq[kb] = *(const FT*)(qp + 32 * kb);
                    } else {
                        const f32x4 x0 = *(const f32x4*)(qp + 32 * kb), x1 = *(const f32x4*)(qp + 32 * kb + 4);
                        fq[kb] = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
                f32x4 qk = {0.f, 0.f, 0.f, 0.f}, kk = qk, dm = qk, da = qk;
#pragma unroll
                for (int kb = 0; kb < VB; ++kb) {
                    const FT f = frag_rows<OT>(ln, vDel, 16 * I, 32 * kb);
                    mma(dm, f, frag_rows<OT>(ln, vO, 16 * R, 32 * kb));
                    mma(da, f, frag_rows<OT>(ln, vDy, 16 * R, 32 * kb));
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const FT f = frag_rows<OT>(ln, vK, 16 * I, 32 * kb);
                    mma(kk, f, frag_rows<OT>(ln, vK, 16 * R, 32 * kb));
                    mma(qk, f, fq[kb]);
                }
                const float rhi = lds_load<float>(hd + LS::VEC + (SC_GHI + r) * 4);
                const float rlo = lds_load<float>(hd + LS::VEC + (SC_GLO + r) * 4);
                const float br = lds_load<float>(hd + LS::VEC + (SC_BETA + r) * 4);
                float ihi[4], ilo[4], nn[4];
                lds_get4<float>(hd + LS::VEC + (SC_GHI + i0) * 4, ihi);
                lds_get4<float>(hd + LS::VEC + (SC_GLO + i0) * 4, ilo);
                float rows = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = i0 + i <= r ? decay<OT>(rhi, rlo, ihi[i], ilo[i]) : 0.f;
                    const bool strict = i0 + i < r;
                    fP[n][i] = d == 0.f ? 0.f : d * dm[i];
                    fRp[n][i] = strict && d != 0.f ? -(d * da[i]) : 0.f;
                    nn[i] = strict ? fP[n][i] * qk[i] + br * fRp[n][i] * kk[i] : 0.f;
                    rows += nn[i];
                }
                rows = sum_lq(rows);
                if (ln.lq == 0) lds_store<float>(sm + LS::ROWP + (p * 16 + ln.li) * 4, rows);
#pragma unroll
                for (int i = 0; i < 4; ++i) nn[i] = row_sum16(nn[i]);
                if (ln.li == 0)
                    lds_store<f32x4>(sm + LS::COLP + (p * 16 + 4 * ln.lq) * 4, f32x4{nn[0], nn[1], nn[2], nn[3]});
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        sync_lds();  // dO, Delta and dY are dead: P and R (and q) take their place
        if (!MULTI) dma_rows_clamped<OT, DK, NW>((const OT*)a.q + k0, rsk, nvalid, hd + LS::QL, wv);
#pragma unroll
        for (int n = 0; n < PPW; ++n) {
            const int p = wv + NW * n;
            if (p < NPAIR) {
                int R, I;
                pair_ri(p, R, I);
                const int o = swz<OT, CH>(16 * R + ln.li, 16 * I + 4 * ln.lq) * ES;
                const float br = lds_load<float>(hd + LS::VEC + (SC_BETA + 16 * R + ln.li) * 4);
                const float x[4] = {fP[n][0], fP[n][1], fP[n][2], fP[n][3]};
                const float y[4] = {fRp[n][0], fRp[n][1], fRp[n][2], fRp[n][3]};
                const float z[4] = {br * y[0], br * y[1], br * y[2], br * y[3]};
                lds_put4<OT>(hd + LS::P + o, x);
                if constexpr (LS::NS == 2) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = x[i] - to_f(to_ot<OT>(x[i]));
                    lds_put4<OT>(hd + LS::PL + o, w);
                }
                lds_put4<OT>(hd + LS::RP + o, y);
                lds_put4<OT>(hd + LS::R + o, z);
            }
        }
        for (int u = wv; u < 6; u += NW) {
            int R, I;
            sc_upper_ri(u, R, I);
            const int o = swz<OT, CH>(16 * R + ln.li, 16 * I + 4 * ln.lq) * ES;
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            lds_put4<OT>(hd + LS::P + o, z);
            if constexpr (LS::NS == 2) lds_put4<OT>(hd + LS::PL + o, z);
            lds_put4<OT>(hd + LS::RP + o, z);
            lds_put4<OT>(hd + LS::R + o, z);
        }
        if (!MULTI) wait_vm<0>();
        sync_lds();

        // ---- dq += P K, G += (R / beta) K, dk += P^T Q + R^T K + beta G
        FT fK[2], fQ[2];
        ln = fresh_lane();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            fK[kb] = frag_cols<OT>(ln, vK, 16 * kw, 32 * kb);
            fQ[kb] = frag_cols<OT>(ln, vQ, 16 * kw, 32 * kb);
        }
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            const int tt = t0 + t;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                if (kb == 0 || tt >= 2) {  // rows of token tile t: columns up to it
                    mma(dq[t], fK[kb], frag_rows<OT>(ln, vP, 16 * tt, 32 * kb));
                    if constexpr (LS::NS == 2) mma(dq[t], fK[kb], frag_rows<OT>(ln, vPl, 16 * tt, 32 * kb));
                    mma(G[t], fK[kb], frag_rows<OT>(ln, vRp, 16 * tt, 32 * kb));
                }
                if (kb == 1 || tt < 2) {   // columns of token tile t: rows from it on
                    mma(dk[t], fQ[kb], frag_cols<OT>(ln, vP, 16 * tt, 32 * kb));
                    if constexpr (LS::NS == 2) mma(dk[t], fQ[kb], frag_cols<OT>(ln, vPl, 16 * tt, 32 * kb));
                    mma(dk[t], fK[kb], frag_cols<OT>(ln, vR, 16 * tt, 32 * kb));
                }
            }
            float kx[4];
            lds_get4<OT>(vK.p + vK.off(16 * tt + ln.li, 16 * kw + 4 * ln.lq), kx);
            dot4(kx, G[t], t, 3);
            dk[t] += G[t] * lds_load<float>(hd + LS::VEC + (SC_BETA + 16 * tt + ln.li) * 4);
            __builtin_amdgcn_sched_barrier(0);
        }
        sync_lds();
        // ---- sums over the waves and over the block pairs, lane = row, one task a wave
        for (int task = wv; task < 6; task += NW) {
            float x = 0.f;
            if (task < 4) {
#pragma unroll
                for (int u = 0; u < KW; ++u) x += lds_load<float>(sm + LS::DOTS + ((task * KW + u) * CH + l) * 4);
            } else if (task == 4) {
                const int b = l / 16;
#pragma unroll
                for (int o = 0; o < NBLK; ++o) {
                    const float rs = lds_load<float>(sm + LS::ROWP + (pair_id(b, min(o, b)) * 16 + l % 16) * 4);
                    const float cs = lds_load<float>(sm + LS::COLP + (pair_id(max(o, b), b) * 16 + l % 16) * 4);
                    x += (o <= b ? rs : 0.f) - (o >= b ? cs : 0.f);
                }
            } else {
#pragma unroll
                for (int u = 0; u < KW; ++u) x += lds_load<float>(sm + LS::SS + u * 4);
            }
            lds_store<float>(sm + LS::RED + (task * CH + l) * 4, x);
        }
        if (!MULTI || hh + 1 == a.R) {  // dq and dk, turned to whole rows through LDS
#pragma unroll
            for (int t = 0; t < TPW; ++t) {
                const int o = swz<OT, DK>(16 * (t0 + t) + ln.li, 16 * kw + 4 * ln.lq) * ES;
                const float x[4] = {dq[t][0], dq[t][1], dq[t][2], dq[t][3]};
                const float y[4] = {dk[t][0], dk[t][1], dk[t][2], dk[t][3]};
                lds_put4<OT>(hd + LS::ODQ + o, x);
                lds_put4<OT>(hd + LS::ODK + o, y);
            }
        }
        sync_lds();
        if (!MULTI || hh + 1 == a.R) {
            store_rows_tiles<OT, DK, NTHR, false>(hd + LS::ODQ, (OT*)a.dq + k0, rsk, nvalid);
            store_rows_tiles<OT, DK, NTHR, false>(hd + LS::ODK, (OT*)a.dk + k0, rsk, nvalid);
        }
        // ---- dbeta and dg
        if (wv == 0) {
            auto red = [&](int t) { return lds_load<float>(sm + LS::RED + (t * CH + l) * 4); };
            const float b = lds_load<float>(hd + LS::VEC + (SC_BETA + l) * 4);
            const float x = red(0) + b * red(1) + red(4);
            // suffix sum of x, exclusive prefix sum of k.dk_s: inside the 16 lanes of a row, then over rows
            float suf = row_suffix16(x), pre = row_scan16(red(2));
            const float s1 = lane_value(suf, 16), s2 = lane_value(suf, 32), s3 = lane_value(suf, 48);
            const float p0 = lane_value(pre, 15), p1 = lane_value(pre, 31), p2 = lane_value(pre, 47);
            pre = row_shr1(pre);
            suf += l < 16 ? s1 + (s2 + s3) : l < 32 ? s2 + s3 : l < 48 ? s3 : 0.f;
            pre += l < 16 ? 0.f : l < 32 ? p0 : l < 48 ? p0 + p1 : (p0 + p1) + p2;
            if (l < nvalid) {
                const size_t at = (size_t)(row0 + l) * a.Hv + h;
                ((OT*)a.dbeta)[at] = to_ot<OT>(lds_load<float>(sm + LS::DOTV + l * 4) + (sc_dbeta_by_delta(b) ? 0.f : red(3)));
                ((OT*)a.dg)[at] = to_ot<OT>(suf + pre + lds_load<float>(hd + LS::VEC + SC_EC * 4) * red(5));
            }
        }
    }
}

// ============================================================================ launchers
template <class OT, int DK, int DV>
static hipError_t launch_sc_fwd_t(const ScArgs& a, bool train, hipStream_t stream) {
    const dim3 grid((unsigned)(a.slots * a.Hv));
    if (train)
        hipLaunchKernelGGL((k_sc_prep<OT, DK, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_sc_prep<OT, DK, false>), grid, dim3(256), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_sc_fwd_chain_t<OT, DK, DV>(a, train, stream);
}
template <class OT, int DK, int DV>
static hipError_t launch_sc_bwd_t(const ScArgs& a, hipStream_t stream) {
    hipError_t e = launch_sc_bwd_chain_t<OT, DK, DV>(a, stream);
    if (e != hipSuccess) return e;
    const int lds = a.R > 1 ? ScGradLds<OT, DK, DV, true>::BYTES : ScGradLds<OT, DK, DV, false>::BYTES;
    auto grad = a.R > 1 ? k_sc_grad<OT, DK, DV, true> : k_sc_grad<OT, DK, DV, false>;
    e = hipFuncSetAttribute((const void*)grad, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grad, dim3((unsigned)(a.slots * a.Hk)), dim3(512), lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_sc_fwd(const ScArgs& a, bool bf16_, bool train, hipStream_t stream) {
    if (bf16_) {
        if (a.DK == 64 && a.DV == 64) return launch_sc_fwd_t<bf16, 64, 64>(a, train, stream);
        if (a.DK == 64 && a.DV == 128) return launch_sc_fwd_t<bf16, 64, 128>(a, train, stream);
        if (a.DK == 128 && a.DV == 64) return launch_sc_fwd_t<bf16, 128, 64>(a, train, stream);
        if (a.DK == 128 && a.DV == 128) return launch_sc_fwd_t<bf16, 128, 128>(a, train, stream);
    } else if (a.DK == 64 && a.DV == 64) {
        return launch_sc_fwd_t<float, 64, 64>(a, train, stream);
    }
    return hipErrorInvalidValue;
}
hipError_t launch_sc_bwd(const ScArgs& a, bool bf16_, hipStream_t stream) {
    if (bf16_) {
        if (a.DK == 64 && a.DV == 64) return launch_sc_bwd_t<bf16, 64, 64>(a, stream);
        if (a.DK == 64 && a.DV == 128) return launch_sc_bwd_t<bf16, 64, 128>(a, stream);
        if (a.DK == 128 && a.DV == 64) return launch_sc_bwd_t<bf16, 128, 64>(a, stream);
        if (a.DK == 128 && a.DV == 128) return launch_sc_bwd_t<bf16, 128, 128>(a, stream);
    } else if (a.DK == 64 && a.DV == 64) {
        return launch_sc_bwd_t<float, 64, 64>(a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace gdr2
