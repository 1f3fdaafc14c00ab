// Attention of one new token over a paged key-value cache on gfx950, and the cache's writer.
//
//     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t - max),   lse = max + log sum_t p_t
//
// over the tokens t of a sequence that lie in its window and on a valid page.
//
// Bound by HBM: every key and value of the window is read once, by one workgroup, for the whole
// group of query heads that share it. The matrix cores take 16 heads (padded) against 16 tokens,
// which costs nothing next to the bytes.
//
// The cache's tokens go straight from memory into matrix operands, without LDS. Keys: a lane of an
// operand fragment holds 8 consecutive channels of one token, which is how they lie in memory. The
// scores come out transposed (rows tokens, columns heads), so that a head's softmax is in one column
// of lanes and its statistics are per-lane scalars; and the fp32 accumulator a lane holds, four
// tokens of its head, is the other product's operand as it is, if that product numbers its tokens
// 4 (lane / 16) + i. Values: a lane loads D / 16 consecutive channels of those same tokens and
// transposes its 8 x 8 block in registers (one byte permute per pair of elements).
//
// Long rows are split evenly over a fixed number of workgroups whatever the lengths: the units (32
// tokens in bf16, 16 in fp32) of all (sequence, head group) rows form one line, with ATTN_COST places
// before each row for what a row costs by itself, and each workgroup takes an equal run of the line,
// its eight waves the units in turn. A row inside one run is finished there; a row that crosses runs
// leaves partial sums, joined in a fixed order by a second kernel. Where no row can be long, each
// workgroup takes one row and there is nothing to join (attn_rows_mode).
//
// Measured: 64 sequences of 200 to 16384 tokens, 32 heads over 8 key heads of 128, bf16 (1.02 GB) 198 us
// with the join, 5.15 TB/s, and 4096 of 300 tokens (5 GB) 1.10 ms, 4.6 TB/s; 24 windows of up to 2048 tokens, 16 heads of 64, fp32 (134 MB)
// 38 us a pass, 3.5 TB/s, of which about 12 us are what even short rows take on the line (two launches,
// the line, the join).
#include "gdr2_attn.hpp"
#include "gdr2_device.hpp"

namespace gdr2 {

template <class OT>
constexpr int attn_unit() { return attn_unit_tokens(sizeof(OT) == 2); }
constexpr int AW = 8;           // waves of a workgroup
constexpr int ATTN_MIN = 14;    // places of the line a workgroup takes at least (ATTN_COST + a unit for each wave)

// The visible tokens of sequence b and its units (at least one, so that every row is written).
struct AttnSpan {
    int lo, hi, u0, units;
};
template <class OT>
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, int b) {
    constexpr int U = attn_unit<OT>();
    const long long cap = (long long)a.c.max_pages << a.c.shift;
    const int len = a.lengths[b];
    AttnSpan s;
    s.hi = len < 0 ? 0 : (long long)len < cap ? len : (int)cap;
    s.lo = a.window > 0 && s.hi > a.window ? s.hi - a.window : 0;
    s.u0 = s.lo / U;
    s.units = max(1, (s.hi + U - 1) / U - s.u0);
    return s;
}

// The line of all rows, computed by each wave for itself: lane t holds the place before its run of
// `per` consecutive sequences. A workgroup takes `share` places. (The host checks that they are fewer
// than 2^31.)
struct AttnLine {
    unsigned before, total, share;
    int per;
};
template <class OT>
__device__ __forceinline__ AttnLine attn_line(const AttnArgs& a) {
    const int l = lane_id(), HR = a.Hkv * a.NG;
    AttnLine p;
    p.per = (a.B + 63) / 64;
    unsigned own = 0;
    for (int i = 0; i < p.per; ++i) {
        const int b = l * p.per + i;
        if (b < a.B) own += (attn_span<OT>(a, b).units + ATTN_COST) * HR;
    }
    unsigned x = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const unsigned y = __shfl_up(x, o);
        if (l >= o) x += y;
    }
    p.before = x - own;
    p.total = __builtin_amdgcn_readlane(x, 63);
    p.share = max((p.total + a.wgs - 1) / a.wgs, (unsigned)ATTN_MIN);
    return p;
}

// The sequence that holds place t (below total): its number, first place and tokens.
struct AttnAt {
    int b;
    unsigned at;
    AttnSpan sp;
};
template <class OT>
__device__ __forceinline__ AttnAt attn_find(const AttnArgs& a, const AttnLine& line, unsigned t) {
    const int HR = a.Hkv * a.NG;
    // the last run of sequences that does not begin behind it, then through that run
    const int ln = __popcll(__ballot(line.before <= t && lane_id() * line.per < a.B)) - 1;
    AttnAt f;
    f.b = ln * line.per;
    f.at = __builtin_amdgcn_readlane(line.before, ln);
    f.sp = attn_span<OT>(a, f.b);
    while (t >= f.at + (f.sp.units + ATTN_COST) * HR) {
        f.at += (f.sp.units + ATTN_COST) * HR;
        f.sp = attn_span<OT>(a, ++f.b);
    }
    return f;
}

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

// pg[s]: page of token tile s of the unit, or negative. Tiles never straddle pages (a page holds a
// multiple of 16 tokens). Invalid tiles read page 0 and are masked.
template <class OT, int D>
__device__ __forceinline__ void attn_load(const AttnArgs& a, int u, int hkv, const int (&pg)[2], AttnTile<OT, D>& t) {
    const int l = lane_id(), li = l & 15, lq = l >> 4;
    constexpr int U = attn_unit<OT>();
    t.ok = 0;
#pragma unroll
    for (int s = 0; s < U / 16; ++s) {
        const int tok = (u * U + 16 * s) & (a.c.page - 1);
        if (pg[s] >= 0) t.ok |= 1 << s;
        const long long page = pg[s] >= 0 ? pg[s] : 0;
        const OT* kp = (const OT*)a.c.k + page * a.c.ks[0] + tok * a.c.ks[1] + hkv * a.c.ks[2];
        const OT* vp = (const OT*)a.c.v + page * a.c.vs[0] + tok * a.c.vs[1] + hkv * a.c.vs[2];
        if constexpr (sizeof(OT) == 2) {
            const OT* kr = kp + li * a.c.ks[1] + 8 * lq;
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) t.k[s][kb] = *(const bf16x8*)(kr + 32 * kb);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t.v[4 * s + i] = *(const typename AttnTile<OT, D>::VT*)(vp + (4 * lq + i) * a.c.vs[1] + (D / 16) * li);
        } else {
            const OT* kr = kp + li * a.c.ks[1] + 4 * lq;
#pragma unroll
            for (int kb = 0; kb < D / 16; ++kb) t.k[kb] = *(const f32x4*)(kr + 16 * kb);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                    t.v[i][j] = *(const f32x4*)(vp + (4 * lq + i) * a.c.vs[1] + (D / 16) * li + 4 * j);
        }
    }
}

// Running softmax of a wave: lane (li, lq) holds head li; l is its own tokens' share of the weight.
// acc[j]: channels (D / 16) (4 lq + i) + j, head li.
template <int D>
struct AttnState {
    float m, l;
    f32x4 acc[D / 16];
};

template <class OT, int D>
__device__ __forceinline__ void attn_update(const AttnArgs& a, const AttnSpan& sp, int u, AttnTile<OT, D>& t,
                                            const typename std::conditional<sizeof(OT) == 2, bf16x8, f32x4>::type* q,
                                            AttnState<D>& st) {
    constexpr int U = attn_unit<OT>(), NS = U / 16, EV = D / 16;
    const int l = lane_id(), lq = l >> 4;
    f32x4 s[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        s[n] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (sizeof(OT) == 2) {
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) mma(s[n], t.k[n][kb], q[kb]);
        } else {
#pragma unroll
            for (int kb = 0; kb < D / 16; ++kb)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(t.k[kb][j], q[kb][j], s[n], 0, 0, 0);
        }
        s[n] = s[n] * a.scale2;
    }
    const int base = u * U;
    if (base < sp.lo || base + U > sp.hi || t.ok != (1 << NS) - 1) {
        // masked tokens: no score, and a zero value, whatever the cache holds there
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = base + 16 * n + 4 * lq + i;
                const bool see = tok >= sp.lo && tok < sp.hi && ((t.ok >> n) & 1);
                s[n][i] = see ? s[n][i] : -INFINITY;
                if constexpr (sizeof(OT) == 2) {
#pragma unroll
                    for (int j = 0; j < EV; ++j) t.v[4 * n + i][j] = see ? t.v[4 * n + i][j] : (bf16)0.f;
                } else {
#pragma unroll
                    for (int j = 0; j < EV / 4; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) t.v[i][j][c] = see ? t.v[i][j][c] : 0.f;
                }
            }
    }
    float mx = s[0][0];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[n][i]);
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(st.m, mx), mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = __builtin_amdgcn_exp2f(st.m - mu);
    st.m = mn;
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[n][i] = __builtin_amdgcn_exp2f(s[n][i] - mu);
            sum += s[n][i];
        }
    st.l = st.l * alpha + sum;
#pragma unroll
    for (int j = 0; j < EV; ++j) st.acc[j] = st.acc[j] * alpha;
    if constexpr (sizeof(OT) == 2) {
        // the weights as two bf16 operands, a value and what its rounding left over: 2^-17 of a weight is lost
        // (one part alone lost up to 2^-8: o was off by 2.1e-3 normwise, where its own rounding is 1.7e-3). The
        // products are still next to nothing beside the bytes: no case took longer.
        bf16x8 p, r;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[4 * n + i] = (bf16)s[n][i];
                r[4 * n + i] = (bf16)(s[n][i] - (float)p[4 * n + i]);
            }
#pragma unroll
        for (int j = 0; j < EV; ++j) {
            bf16x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = t.v[e][j];
            mma(st.acc[j], v, p);
            mma(st.acc[j], v, r);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < EV; ++j)
                st.acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(t.v[i][j / 4][j % 4], s[0][i], st.acc[j], 0, 0, 0);
    }
}

// One run of a row by the workgroup's waves: units i0 .. i0 + n - 1 of the row's; whole: the whole row,
// finished here, else its partial sums go to `part`.
template <class OT, int D>
__device__ __forceinline__ void attn_run(const AttnArgs& a, int b, int hr, const AttnSpan& sp, int i0, int n, bool whole,
                                         float* part, float (&sml)[2][AW][16], float (&so)[AW][16][D + 4]) {
    constexpr int U = attn_unit<OT>(), EV = D / 16;
    using QT = typename std::conditional<sizeof(OT) == 2, bf16x8, f32x4>::type;
    constexpr int NQ = sizeof(OT) == 2 ? D / 32 : D / 16;
    const int tid = threadIdx.x, l = tid & 63, li = l & 15, lq = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hkv = hr / a.NG, h0 = hkv * a.G + (hr % a.NG) * a.gh;  // first query head of the row
    const int heads = min(a.gh, a.G - (hr % a.NG) * a.gh);
    const int u0 = sp.u0 + i0;
    const int work = sp.hi > sp.lo ? n : 0;  // a row with nothing to see has a unit, but no page to read
    auto pages = [&](int i, int (&pg)[2]) {  // pages of unit i of the run
#pragma unroll
        for (int s = 0; s < U / 16; ++s) {
            const int tok = (u0 + i) * U + 16 * s;
            pg[s] = -1;
            if (i < work && tok < sp.hi) {
                const int p = a.c.table[(size_t)b * a.c.max_pages + (tok >> a.c.shift)];
                pg[s] = (unsigned)p < (unsigned)a.c.pages ? p : -1;
            }
        }
    };
    int pg[2] = {-1, -1};
    pages(wv, pg);
    QT q[NQ];
    {
        const OT* qp = (const OT*)a.q + ((size_t)b * a.Hq + h0 + min(li, heads - 1)) * D;
#pragma unroll
        for (int kb = 0; kb < NQ; ++kb) {
            if constexpr (sizeof(OT) == 2) q[kb] = *(const QT*)(qp + 32 * kb + 8 * lq);
            else q[kb] = *(const QT*)(qp + 16 * kb + 4 * lq);
        }
    }
    AttnState<D> st;
    st.m = -INFINITY;
    st.l = 0.f;
#pragma unroll
    for (int j = 0; j < EV; ++j) st.acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the wave's units wv, wv + AW, ..: the next one's keys and values are on their way while this one
    // is worked on, and the page of the one after that is looked up
    AttnTile<OT, D> t0, t1;
    if (wv < work) {
        attn_load<OT, D>(a, u0 + wv, hkv, pg, t0);
        pages(wv + AW, pg);
    }
#pragma unroll 1
    for (int i = wv; i < work; i += 2 * AW) {
        if (i + AW < work) {
            attn_load<OT, D>(a, u0 + i + AW, hkv, pg, t1);
            pages(i + 2 * AW, pg);
        }
        attn_update<OT, D>(a, sp, u0 + i, t0, q, st);
        if (i + AW >= work) break;
        if (i + 2 * AW < work) {
            attn_load<OT, D>(a, u0 + i + 2 * AW, hkv, pg, t0);
            pages(i + 3 * AW, pg);
        }
        attn_update<OT, D>(a, sp, u0 + i + AW, t1, q, st);
    }
    // ---- join the waves
    st.l += __shfl_xor(st.l, 16);
    st.l += __shfl_xor(st.l, 32);
    if (lq == 0) {
        sml[0][wv][li] = st.m;
        sml[1][wv][li] = st.l;
    }
    __syncthreads();
    float M = sml[0][0][li];
#pragma unroll
    for (int x = 1; x < AW; ++x) M = fmaxf(M, sml[0][x][li]);
    const float f = __builtin_amdgcn_exp2f(st.m - (M == -INFINITY ? 0.f : M));
    if (li < heads) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j4 = 0; j4 < EV; j4 += 4) {
                f32x4 x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = st.acc[j4 + j][i] * f;
                *(f32x4*)&so[wv][li][EV * (4 * lq + i) + j4] = x;
            }
    }
    __syncthreads();
    for (int e = tid; e < heads * (D / 4); e += 64 * AW) {
        const int hd = e / (D / 4), d = 4 * (e % (D / 4));
        f32x4 x = *(const f32x4*)&so[0][hd][d];
#pragma unroll
        for (int y = 1; y < AW; ++y) x += *(const f32x4*)&so[y][hd][d];
        float Mh = sml[0][0][hd];
#pragma unroll
        for (int y = 1; y < AW; ++y) Mh = fmaxf(Mh, sml[0][y][hd]);
        const float mu = Mh == -INFINITY ? 0.f : Mh;
        float L = 0.f;
#pragma unroll
        for (int y = 0; y < AW; ++y) L += sml[1][y][hd] * __builtin_amdgcn_exp2f(sml[0][y][hd] - mu);
        if (whole) {
            const float r = L == 0.f ? 0.f : 1.f / L;  // nothing visible: a row of zeros
            const float ov[4] = {x[0] * r, x[1] * r, x[2] * r, x[3] * r};
            st4((OT*)a.o + ((size_t)b * a.Hq + h0 + hd) * D + d, ov);
            if (a.lse && d == 0)
                a.lse[(size_t)b * a.Hq + h0 + hd] = L == 0.f ? -INFINITY : (Mh + __log2f(L)) * 0.6931471805599453f;
        } else {
            *(f32x4*)(part + (size_t)hd * D + d) = x;
            if (d == 0) {
                part[(size_t)a.gh * D + 2 * hd] = Mh;
                part[(size_t)a.gh * D + 2 * hd + 1] = L;
            }
        }
    }
}

// SPLIT: the line of rows, an equal run a workgroup; else one row a workgroup.
template <class OT, int D, bool SPLIT>
__global__ __launch_bounds__(64 * AW) void k_attn(AttnArgs a) {
    __shared__ float sml[2][AW][16];
    __shared__ __align__(16) float so[AW][16][D + 4];
    poison_lds((lds_char*)sml, sizeof(sml));
    poison_lds((lds_char*)so, sizeof(so));
    poison_lds_done();
    const int HR = a.Hkv * a.NG;  // rows of a sequence
    if constexpr (!SPLIT) {
        const int b = blockIdx.x / HR, hr = blockIdx.x % HR;
        const AttnSpan sp = attn_span<OT>(a, b);
        attn_run<OT, D>(a, b, hr, sp, 0, sp.units, true, nullptr, sml, so);
        return;
    }
    const AttnLine line = attn_line<OT>(a);
    unsigned t = blockIdx.x * line.share;
    if (t >= line.total) return;
    const unsigned tend = min(t + line.share, line.total);
    AttnAt f = attn_find<OT>(a, line, t);
    int b = f.b;
    unsigned at = f.at;
    AttnSpan sp = f.sp;
    while (t < tend) {
        const int len = sp.units + ATTN_COST;
        const int hr = (t - at) / len;
        const unsigned r0 = at + (unsigned)hr * len;             // the row's first place
        const unsigned r1 = min(r0 + len, tend);
        // its units in this run: place r0 + ATTN_COST + i is unit i
        const int i0 = max(0, (int)(t - r0) - ATTN_COST), i1 = max(0, (int)(r1 - r0) - ATTN_COST);
        if (i1 > i0) {
            const bool whole = i1 - i0 == sp.units;
            // a row that goes on from the workgroup before leaves its sums in slot 0, one that begins
            // here and goes on in slot 1: there is at most one of each
            float* part = a.part + (size_t)(2 * blockIdx.x + (i0 > 0 ? 0 : 1)) * ((size_t)a.gh * (D + 4));
            attn_run<OT, D>(a, b, hr, sp, i0, i1 - i0, whole, part, sml, so);
            __syncthreads();
        }
        t = r1;
        if (t < tend && t == at + (unsigned)len * HR) {
            at = t;
            sp = attn_span<OT>(a, ++b);
        }
    }
}

// Joins the partial results of the rows that cross workgroups, the workgroups' parts of a row in order. One
// workgroup for each run of the line but the last and each head of a group: at most one row begins in a run
// and goes on behind it. (With one for each row, each of which walked the line, 4096 sequences took 4.9 ms.)
template <class OT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    constexpr int NGRP = 256 / (D / 4);  // thread groups over the parts
    __shared__ float sM[NGRP], sL[NGRP];
    __shared__ __align__(16) float so[NGRP][D];
    poison_lds((lds_char*)sM, sizeof(sM));
    poison_lds((lds_char*)sL, sizeof(sL));
    poison_lds((lds_char*)so, sizeof(so));
    poison_lds_done();
    const int tid = threadIdx.x;
    const unsigned w0 = blockIdx.x / a.gh;
    const int hd = blockIdx.x % a.gh;
    const AttnLine line = attn_line<OT>(a);
    const unsigned t = (w0 + 1) * line.share;  // the first place behind the run
    if (t >= line.total) return;
    const AttnAt f = attn_find<OT>(a, line, t);
    const int b = f.b, len = f.sp.units + ATTN_COST, hr = (t - f.at) / len;
    const unsigned r0 = f.at + (unsigned)hr * len + ATTN_COST;  // the place of the row's unit 0
    if (r0 >= t || r0 / line.share != w0) return;  // it begins behind the run, or before it
    const unsigned w1 = (r0 + f.sp.units - 1) / line.share;
    const int hkv = hr / a.NG, hg = (hr % a.NG) * a.gh + hd;
    if (hg >= a.G) return;
    const int hq = hkv * a.G + hg;
    const size_t stride = (size_t)a.gh * (D + 4);
    const int g = tid / (D / 4), d = 4 * (tid % (D / 4));
    float M = -INFINITY, L = 0.f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    for (unsigned w = w0 + g; w <= w1; w += NGRP) {
        const float* p = a.part + (size_t)(2 * w + (w == w0 ? 1 : 0)) * stride;
        const float m = p[(size_t)a.gh * D + 2 * hd], lw = p[(size_t)a.gh * D + 2 * hd + 1];
        const f32x4 y = *(const f32x4*)(p + (size_t)hd * D + d);
        const float mn = fmaxf(M, m), mu = mn == -INFINITY ? 0.f : mn;
        const float fa = __builtin_amdgcn_exp2f(M - mu), fb = __builtin_amdgcn_exp2f(m - mu);
        x = x * fa + y * fb;
        L = L * fa + lw * fb;
        M = mn;
    }
    *(f32x4*)&so[g][d] = x;
    if (d == 0) {
        sM[g] = M;
        sL[g] = L;
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int i = 1; i < NGRP; ++i) M = fmaxf(M, sM[i]);
        const float mu = M == -INFINITY ? 0.f : M;
        L = 0.f;
        x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NGRP; ++i) {
            const float f = __builtin_amdgcn_exp2f(sM[i] - mu);
            L += sL[i] * f;
            x += *(const f32x4*)&so[i][d] * f;
        }
        const float r = L == 0.f ? 0.f : 1.f / L;
        const float ov[4] = {x[0] * r, x[1] * r, x[2] * r, x[3] * r};
        st4((OT*)a.o + ((size_t)b * a.Hq + hq) * D + d, ov);
        if (a.lse && d == 0)
            a.lse[(size_t)b * a.Hq + hq] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
    }
}

// One row a workgroup, without a second kernel: where the table (or the window) leaves a row at most four
// units for each wave, 1024 tokens in bf16. Measured in a graph, bf16, 4 key heads of 128, one row a
// workgroup against the line of runs and its join:
//   1 sequence of 100 tokens   4.7 and 11.7 us     1 of 777   11.4 and 13.8     1 of 2048   22.4 and 14.0
//   8 of 1000                 18.4 and 16.7       32 of 1000  20.8 and 22.9    32 of 2048   40.1 and 36.2
//   200 of 500                53.3 and 56.8      200 of 2048 174.7 and 162.5  200 of 4096  340.4 and 305.3
// (the last 5.5 TB/s; long rows one a workgroup leave compute units idle at the end). A launch takes fewer than
// 2^32 threads: 2^23 rows and more go to the line.
inline bool attn_rows_mode(const AttnArgs& a, int unit) {
    const long long rows = (long long)a.B * a.Hkv * a.NG;
    return attn_max_units(a.c, a.window, unit) <= 4 * AW && rows < (1LL << 32) / (64 * AW);
}

template <class OT, int D>
static hipError_t launch_attn_t(const AttnArgs& a, hipStream_t stream) {
    if (attn_rows_mode(a, attn_unit<OT>())) {
        hipLaunchKernelGGL((k_attn<OT, D, false>), dim3((unsigned)(a.B * a.Hkv * a.NG)), dim3(64 * AW), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_attn<OT, D, true>), dim3(a.wgs), dim3(64 * AW), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attn_join<OT, D>), dim3((unsigned)((a.wgs - 1) * a.gh)), dim3(256), 0, stream, a);
    return hipGetLastError();
}
hipError_t launch_attn(const AttnArgs& a, bool bf16_, hipStream_t stream) {
    if (bf16_) return a.D == 64 ? launch_attn_t<bf16, 64>(a, stream) : launch_attn_t<bf16, 128>(a, stream);
    return a.D == 64 ? launch_attn_t<float, 64>(a, stream) : launch_attn_t<float, 128>(a, stream);
}

// ============================================================================ writing the cache
// Bound by HBM: 56 MB of prompts in 11.8 us, 4.7 TB/s; one token for each of 96 sequences 2.9 us, a launch.
// A copy, 16 bytes a thread for the keys and the values each; a token's row (all its heads) by
// consecutive threads. Tokens whose place lies past the table or on an invalid page are dropped.
template <class OT>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
    constexpr int EPC = 16 / (int)sizeof(OT);
    const int hc = a.D / EPC, nch = a.Hkv * hc;  // 16-byte pieces of a head and of a token's row
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long tok = e / nch;
    if (tok >= a.tokens) return;
    const int ch = (int)(e % nch), h = ch / hc, d = EPC * (ch % hc);
    int s = (int)tok;
    long long off = 0;
    if (a.cu) {
        int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before the token
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (a.cu[mid] <= tok) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        if (tok < a.cu[s] || tok >= a.cu[s + 1]) return;  // before the first or behind the last sequence
        off = tok - a.cu[s];
    }
    const long long pos = a.starts[s] + off;
    if (pos < 0 || (pos >> a.c.shift) >= a.c.max_pages) return;
    const int page = a.c.table[(size_t)s * a.c.max_pages + (pos >> a.c.shift)];
    if ((unsigned)page >= (unsigned)a.c.pages) return;
    const long long in = pos & (a.c.page - 1);
    const size_t src = (size_t)tok * a.Hkv * a.D + (size_t)h * a.D + d;
    const f32x4 k = *(const f32x4*)((const OT*)a.k + src), v = *(const f32x4*)((const OT*)a.v + src);
    *(f32x4*)((OT*)a.c.k + page * a.c.ks[0] + in * a.c.ks[1] + h * a.c.ks[2] + d) = k;
    *(f32x4*)((OT*)a.c.v + page * a.c.vs[0] + in * a.c.vs[1] + h * a.c.vs[2] + d) = v;
}

hipError_t launch_append(const AppendArgs& a, bool bf16_, hipStream_t stream) {
    const long long n = (long long)a.tokens * a.Hkv * (a.D / (bf16_ ? 8 : 4));
    const dim3 grid((unsigned)((n + 255) / 256));
    if (bf16_)
        hipLaunchKernelGGL((k_append<bf16>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_append<float>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdr2
