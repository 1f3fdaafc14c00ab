// Attention of a tree of drafted tokens over a paged key-value cache on gfx950, and the move that keeps an accepted
// path of the tree.
//
//     o_i = sum_t p_it v_t / sum_t p_it,   p_it = exp(scale q_i.k_t - max),   lse_i = max + log sum_t p_it
//
// over the tokens t that draft i sees: the context that its sequence holds, the drafts above it in the tree, itself.
//
// Bound by HBM as the step of one token (gdr2_attn.hip), whose way of going from the cache into matrix operands
// without LDS it shares. The columns of the products are (draft, head) pairs: a wave takes up to 32 of them against
// each unit of tokens, and where there are more, waves side by side take the same unit, which only the first of them
// brings in from far. A draft's mask is one 64-bit number, the drafts above it, which every wave works out for itself
// from the parents (each round of lane exchanges doubles the way up that is known); only units that reach into the
// drafts, or a window's edge, look at it. Rows are split over workgroups as in gdr2_attn.hip.
//
// Measured with the join, 6 drafts, 32 heads over 8 of 128: 64 sequences of 4000 tokens 198 us in bf16 (1.05 GB, 5.3 TB/s) and 410
// in fp32 (5.1 TB/s); one of 4000 26 and 33 us, two kernels' latency.
#include "gdr2_attn_device.hpp"
#include "gdr2_tree_device.hpp"

namespace gdr2 {

// Running softmax of a wave's columns: lane (li, lq) holds column 16 n + li; l is its own tokens' share of the weight.
// acc[n][j]: channels (D / 16) (4 lq + i) + j. lo, sees: the column's mask.
template <int D, int NC>
struct TreeState {
    float m[NC], l[NC];
    f32x4 acc[NC][D / 16];
    int lo[NC];
    unsigned long long sees[NC];
};

template <class OT, int D, int NC>
__device__ __forceinline__ void tree_run(const TreeArgs& a, int b, int hr, const TreeSpan& sp, int i0, int n, bool whole,
                                         float* part, float (&sml)[2][AW][16 * NC], float (&so)[AW][16 * NC][D + 4]) {
    constexpr int U = attn_unit<OT>(), NS = U / 16, EV = D / 16;
    using QT = typename std::conditional<sizeof(OT) == 2, bf16x8, f32x4>::type;
    constexpr int NQ = sizeof(OT) == 2 ? D / 32 : D / 16;
    const int tid = threadIdx.x, l = tid & 63, li = l & 15, lq = l >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rgi = wv & (a.rg - 1), ks = wv / a.rg, KS = AW / a.rg;  // the wave's columns; its share of the units
    const int hkv = hr / a.nb, blk = hr % a.nb, rows = a.T * a.G;
    const int c0 = (blk * a.rg + rgi) * 16 * NC;
    const int u0 = sp.u0 + i0;
    const int work = sp.hi > sp.lo ? n : 0;  // a row with nothing to see has a unit, but no page to read
    int pg[2], pn[2];
    attn_pages<OT>(a.c, b, u0 + ks, sp.hi, ks < work, pg);
    QT q[NC][NQ];
    TreeState<D, NC> st;
    const TreeLane tl = tree_lane(a, b);
    bool one[NC];
#pragma unroll
    for (int x = 0; x < NC; ++x) {
        const int c = min(c0 + 16 * x + li, rows - 1), i = c / a.G, g = c % a.G;
        const OT* qp = (const OT*)a.q + (((size_t)b * a.T + i) * a.Hq + hkv * a.G + g) * D;
#pragma unroll
        for (int kb = 0; kb < NQ; ++kb) {
            if constexpr (sizeof(OT) == 2) q[x][kb] = *(const QT*)(qp + 32 * kb + 8 * lq);
            else q[x][kb] = *(const QT*)(qp + 16 * kb + 4 * lq);
        }
        st.m[x] = -INFINITY;
        st.l[x] = 0.f;
#pragma unroll
        for (int j = 0; j < EV; ++j) st.acc[x][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        st.sees[x] = __shfl(tl.sees, i);
        const int dep = __shfl(tl.depth, i);
        one[x] = (tl.all >> i) & 1;
        st.lo[x] = !one[x] ? 0x7fffffff : a.window > 0 ? (int)max(0ll, (long long)sp.start + dep + 1 - a.window) : 0;
    }
    // first token that the deepest draft sees
    const int lo_in = a.window > 0 ? (int)max(0ll, (long long)sp.start + a.T - a.window) : 0;
    AttnTile<OT, D> t;
    attn_ok<OT, D>(pg, t);
    if (ks < work) {
        attn_load_k<OT, D>(a.c, u0 + ks, hkv, pg, t);
        attn_load_v<OT, D>(a.c, u0 + ks, hkv, pg, t);
    }
    attn_pages<OT>(a.c, b, u0 + ks + KS, sp.hi, ks + KS < work, pn);
#pragma unroll 1
    for (int i = ks; i < work; i += KS) {
        const int base = (u0 + i) * U, okp = t.ok;
        f32x4 s[NC][NS];
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                s[x][m] = f32x4{0.f, 0.f, 0.f, 0.f};
                if constexpr (sizeof(OT) == 2) {
#pragma unroll
                    for (int kb = 0; kb < NQ; ++kb) mma(s[x][m], t.k[m][kb], q[x][kb]);
                } else {
#pragma unroll
                    for (int kb = 0; kb < NQ; ++kb)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s[x][m] = __builtin_amdgcn_mfma_f32_16x16x4f32(t.k[kb][j], q[x][kb][j], s[x][m], 0, 0, 0);
                }
                s[x][m] = s[x][m] * a.scale2;
            }
        // the next unit's keys are on their way while this one's weights and values are worked on, its values
        // while the next one's scores are
        const bool more = i + KS < work;
        if (more) {
            attn_load_k<OT, D>(a.c, u0 + i + KS, hkv, pn, t);
            attn_ok<OT, D>(pn, t);
        }
        if (base < lo_in || base + U > sp.start || okp != (1 << NS) - 1) {
#pragma unroll
            for (int m = 0; m < NS; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = base + 16 * m + 4 * lq + j, dr = tok - sp.start;
                    const bool in = tok >= sp.lo && tok < sp.hi && ((okp >> m) & 1);
#pragma unroll
                    for (int x = 0; x < NC; ++x) {
                        const bool see = in && (dr < 0 ? tok >= st.lo[x] : (bool)((st.sees[x] >> (dr & 63)) & 1));
                        s[x][m][j] = see ? s[x][m][j] : -INFINITY;
                    }
                    // what no draft sees has a zero value, whatever the cache holds there
                    const bool any = in && (dr < 0 || ((tl.all >> (dr & 63)) & 1));
                    if constexpr (sizeof(OT) == 2) {
#pragma unroll
                        for (int c = 0; c < EV; ++c) t.v[4 * m + j][c] = any ? t.v[4 * m + j][c] : (bf16)0.f;
                    } else {
#pragma unroll
                        for (int c = 0; c < EV; ++c) t.v[j][c / 4][c % 4] = any ? t.v[j][c / 4][c % 4] : 0.f;
                    }
                }
        }
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            float mx = s[x][0][0];
#pragma unroll
            for (int m = 0; m < NS; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) mx = fmaxf(mx, s[x][m][j]);
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = fmaxf(st.m[x], mx), mu = mn == -INFINITY ? 0.f : mn;
            const float alpha = __builtin_amdgcn_exp2f(st.m[x] - mu);
            st.m[x] = mn;
            float sum = 0.f;
#pragma unroll
            for (int m = 0; m < NS; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[x][m][j] = __builtin_amdgcn_exp2f(s[x][m][j] - mu);
                    sum += s[x][m][j];
                }
            st.l[x] = st.l[x] * alpha + sum;
#pragma unroll
            for (int j = 0; j < EV; ++j) st.acc[x][j] = st.acc[x][j] * alpha;
        }
        if constexpr (sizeof(OT) == 2) {
            // weights in two bf16 parts, as in gdr2_attn.hip
            bf16x8 p[NC], r[NC];
#pragma unroll
            for (int x = 0; x < NC; ++x)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[x][4 * m + j] = (bf16)s[x][m][j];
                        r[x][4 * m + j] = (bf16)(s[x][m][j] - (float)p[x][4 * m + j]);
                    }
#pragma unroll
            for (int j = 0; j < EV; ++j) {
                bf16x8 v;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = t.v[e][j];
#pragma unroll
                for (int x = 0; x < NC; ++x) {
                    mma(st.acc[x][j], v, p[x]);
                    mma(st.acc[x][j], v, r[x]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < EV; ++c)
#pragma unroll
                    for (int x = 0; x < NC; ++x)
                        st.acc[x][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(t.v[j][c / 4][c % 4], s[x][0][j], st.acc[x][c], 0, 0, 0);
        }
        if (more) attn_load_v<OT, D>(a.c, u0 + i + KS, hkv, pn, t);
        attn_pages<OT>(a.c, b, u0 + i + 2 * KS, sp.hi, i + 2 * KS < work, pn);
    }
    // ---- join the waves of the same columns
#pragma unroll
    for (int x = 0; x < NC; ++x) {
        st.l[x] += __shfl_xor(st.l[x], 16);
        st.l[x] += __shfl_xor(st.l[x], 32);
        if (!one[x]) {  // padding sees nothing
            st.l[x] = 0.f;
            st.m[x] = -INFINITY;
        }
        if (lq == 0) {
            sml[0][wv][16 * x + li] = st.m[x];
            sml[1][wv][16 * x + li] = st.l[x];
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NC; ++x) {
        float M = -INFINITY;
        for (int y = 0; y < KS; ++y) M = fmaxf(M, sml[0][y * a.rg + rgi][16 * x + li]);
        const float f = __builtin_amdgcn_exp2f(st.m[x] - (M == -INFINITY ? 0.f : M));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j4 = 0; j4 < EV; j4 += 4) {
                f32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = one[x] ? st.acc[x][j4 + j][i] * f : 0.f;
                *(f32x4*)&so[wv][16 * x + li][EV * (4 * lq + i) + j4] = y;
            }
    }
    __syncthreads();
    const int per = 16 * NC * a.rg;  // rows of a block
    for (int e = tid; e < per * (D / 4); e += 64 * AW) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4)), w0 = r / (16 * NC), rc = r % (16 * NC);
        const int c = blk * per + r;
        if (c >= rows) continue;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        float M = -INFINITY, L = 0.f;
        for (int y = 0; y < KS; ++y) {
            x += *(const f32x4*)&so[y * a.rg + w0][rc][d];
            M = fmaxf(M, sml[0][y * a.rg + w0][rc]);
        }
        const float mu = M == -INFINITY ? 0.f : M;
        for (int y = 0; y < KS; ++y)
            L += sml[1][y * a.rg + w0][rc] * __builtin_amdgcn_exp2f(sml[0][y * a.rg + w0][rc] - mu);
        if (whole) {
            const size_t row = ((size_t)b * a.T + c / a.G) * a.Hq + hkv * a.G + c % a.G;
            const float f = L == 0.f ? 0.f : 1.f / L;  // nothing visible: a row of zeros
            const float ov[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
            st4((OT*)a.o + row * D + d, ov);
            if (a.lse && d == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
        } else {
            *(f32x4*)(part + (size_t)r * D + d) = x;
            if (d == 0) {
                part[(size_t)per * D + 2 * r] = M;
                part[(size_t)per * D + 2 * r + 1] = L;
            }
        }
    }
}

// SPLIT: the line of rows, an equal run a workgroup; else one row a workgroup.
template <class OT, int D, int NC, bool SPLIT>
__global__ __launch_bounds__(64 * AW) void k_tree(TreeArgs a) {
    extern __shared__ __align__(16) char smem[];
    float (&so)[AW][16 * NC][D + 4] = *(float (*)[AW][16 * NC][D + 4])smem;
    __shared__ float sml[2][AW][16 * NC];
    poison_lds((lds_char*)smem, sizeof(so));
    poison_lds((lds_char*)sml, sizeof(sml));
    poison_lds_done();
    const int HR = a.Hkv * a.nb;
    if constexpr (!SPLIT) {
        const int b = blockIdx.x / HR, hr = blockIdx.x % HR;
        const TreeSpan sp = tree_span<attn_unit<OT>()>(a, b);
        tree_run<OT, D, NC>(a, b, hr, sp, 0, sp.units, true, nullptr, sml, so);
        return;
    }
    const TreeLine line = tree_line<attn_unit<OT>()>(a);
    unsigned t = blockIdx.x * line.share;
    if (t >= line.total) return;
    const unsigned tend = min(t + line.share, line.total);
    TreeAt f = tree_find<attn_unit<OT>()>(a, line, t);
    int b = f.b;
    unsigned at = f.at;
    TreeSpan sp = f.sp;
    while (t < tend) {
        const int len = sp.units + a.cost;
        const int hr = (t - at) / len;
        const unsigned r0 = at + (unsigned)hr * len;
        const unsigned r1 = min(r0 + len, tend);
        const int i0 = max(0, (int)(t - r0) - a.cost), i1 = max(0, (int)(r1 - r0) - a.cost);
        if (i1 > i0) {
            const bool whole = i1 - i0 == sp.units;
            float* part = a.part + (size_t)(2 * blockIdx.x + (i0 > 0 ? 0 : 1)) * ((size_t)16 * NC * a.rg * (D + 4));
            tree_run<OT, D, NC>(a, b, hr, sp, i0, i1 - i0, whole, part, sml, so);
            __syncthreads();
        }
        t = r1;
        if (t < tend && t == at + (unsigned)len * HR) {
            at = t;
            sp = tree_span<attn_unit<OT>()>(a, ++b);
        }
    }
}

// Joins the rows that cross workgroups, the parts of each in order. Workgroup (w0, y): the row that begins in run w0
// and goes on behind it, if there is one, and of its block's (draft, head) rows y, y + gridDim.y, ..
template <class OT, int D>
__global__ __launch_bounds__(256) void k_tree_join(TreeArgs a) {
    constexpr int NGRP = 256 / (D / 4);
    __shared__ float sM[NGRP], sL[NGRP];
    __shared__ __align__(16) float so[NGRP][D];
    poison_lds((lds_char*)sM, sizeof(sM));
    poison_lds((lds_char*)sL, sizeof(sL));
    poison_lds((lds_char*)so, sizeof(so));
    poison_lds_done();
    const int tid = threadIdx.x;
    const unsigned w0 = blockIdx.x;
    const TreeLine line = tree_line<attn_unit<OT>()>(a);
    const unsigned t = (w0 + 1) * line.share;  // the first place behind the run
    if (t >= line.total) return;
    const TreeAt f = tree_find<attn_unit<OT>()>(a, line, t);
    const int len = f.sp.units + a.cost, hr = (t - f.at) / len;
    const unsigned r0 = f.at + (unsigned)hr * len + a.cost;  // the place of the row's unit 0
    if (r0 >= t || r0 / line.share != w0) return;
    const unsigned w1 = (r0 + f.sp.units - 1) / line.share;
    const int hkv = hr / a.nb, per = 16 * a.nc * a.rg, c0 = hr % a.nb * per;
    const size_t stride = (size_t)per * (D + 4);
    const int g = tid / (D / 4), d = 4 * (tid % (D / 4));
    for (int r = blockIdx.y; r < per && c0 + r < a.T * a.G; r += gridDim.y) {
        float M = -INFINITY, L = 0.f;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (unsigned w = w0 + g; w <= w1; w += NGRP) {
            const float* p = a.part + (size_t)(2 * w + (w == w0 ? 1 : 0)) * stride;
            const float m = p[(size_t)per * D + 2 * r], lw = p[(size_t)per * D + 2 * r + 1];
            const f32x4 y = *(const f32x4*)(p + (size_t)r * D + d);
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
                const float fi = __builtin_amdgcn_exp2f(sM[i] - mu);
                L += sL[i] * fi;
                x += *(const f32x4*)&so[i][d] * fi;
            }
            const int c = c0 + r;
            const size_t row = ((size_t)f.b * a.T + c / a.G) * a.Hq + hkv * a.G + c % a.G;
            const float fl = L == 0.f ? 0.f : 1.f / L;
            const float ov[4] = {x[0] * fl, x[1] * fl, x[2] * fl, x[3] * fl};
            st4((OT*)a.o + row * D + d, ov);
            if (a.lse && d == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// One row a workgroup, without a second kernel, where no row can pass four units a wave (as gdr2_attn.hip). Us, so and on the
// line, 6 drafts, 32 heads over 8 of 128: 1 x 777 tokens 16.2 and 25.6, 64 x 777 42 and 50; with eight units 1 x 1500 22.9 and 25.9,
// 64 x 1500 84 and 90, but 1 x 2000 27.0 and 25.3 (4 drafts, 16 heads over 4 23.9 and 17.6), 8 x 2000 25.7 and 21.8; fp32, units half
// as long: 1 x 480 29.3 and 30.5, 64 x 480 64 and 74; with eight units 1 x 777 41 and 31, 64 x 777 94 and 106.
inline bool tree_rows_mode(const TreeArgs& a) {
    const long long rows = (long long)a.B * a.Hkv * a.nb;
    return tree_max_units(a) <= 4 * (AW / a.rg) && rows < (1LL << 32) / (64 * AW);
}

template <class OT, int D, int NC>
static hipError_t launch_tree_t(const TreeArgs& a, hipStream_t stream) {
    constexpr int LDS = AW * 16 * NC * (D + 4) * 4;
    const auto one = k_tree<OT, D, NC, false>, line = k_tree<OT, D, NC, true>;
    const bool rows = tree_rows_mode(a);
    if (LDS > 65536 - 4096) {
        const hipError_t e = hipFuncSetAttribute(rows ? (const void*)one : (const void*)line,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) return e;
    }
    if (rows) {
        hipLaunchKernelGGL(one, dim3((unsigned)(a.B * a.Hkv * a.nb)), dim3(64 * AW), LDS, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(line, dim3(a.wgs), dim3(64 * AW), LDS, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int per = 16 * a.nc * a.rg;
    hipLaunchKernelGGL((k_tree_join<OT, D>), dim3((unsigned)(a.wgs - 1), (unsigned)(per < 16 ? per : 16)), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <class OT, int D>
static hipError_t launch_tree_d(const TreeArgs& a, hipStream_t stream) {
    return a.nc == 1 ? launch_tree_t<OT, D, 1>(a, stream) : launch_tree_t<OT, D, 2>(a, stream);
}
hipError_t launch_tree(const TreeArgs& a, bool bf16_, hipStream_t stream) {
    if (a.wide) return launch_tree_wide(a, stream);
    if (bf16_) return a.D == 64 ? launch_tree_d<bf16, 64>(a, stream) : launch_tree_d<bf16, 128>(a, stream);
    return a.D == 64 ? launch_tree_d<float, 64>(a, stream) : launch_tree_d<float, 128>(a, stream);
}

// ============================================================================ keeping an accepted path
// Token starts + path[j] of a sequence goes to starts + j, for the entries before its first negative one. A workgroup
// takes 16 pieces of 16 bytes of a token's row, of all (at most 64) tokens, and reads them all before it writes any:
// whatever the path's order, no token is read after another one took its place.
__global__ __launch_bounds__(256) void k_keep(KeepArgs a) {
    const int hc = a.D * a.es / 16, nch = a.Hkv * hc;  // 16-byte pieces of a head and of a token's row
    const int groups = nch > 0 ? (nch + 15) / 16 : 1, b = blockIdx.x / groups, g = blockIdx.x % groups;
    const int l = lane_id();
    const long long st = a.starts[b];
    const int src = l < a.P ? a.path[(size_t)b * a.P + l] : -1;
    const unsigned long long end = __ballot(src < 0);
    const int n = end ? (int)__builtin_ctzll(end) : 64;
    if (a.lengths && g == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.lengths[b] = (int)(st + n);
    const int piece = 16 * g + (threadIdx.x & 15), h = piece / hc;
    const long long* sd = blockIdx.y ? a.c.vs : a.c.ks;
    char* base = (char*)(blockIdx.y ? a.c.v : a.c.k);
    f32x4 x[4];
    char* to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = 16 * i + (threadIdx.x >> 4);
        to[i] = nullptr;
        const int from = __shfl(src, j);
        if (j < n && piece < nch && from != j) {
            auto place = [&](long long pos) -> char* {
                if (pos < 0 || (pos >> a.c.shift) >= a.c.max_pages) return nullptr;
                const int pg = a.c.table[(size_t)b * a.c.max_pages + (pos >> a.c.shift)];
                if ((unsigned)pg >= (unsigned)a.c.pages) return nullptr;
                return base + (pg * sd[0] + (pos & (a.c.page - 1)) * sd[1] + h * sd[2]) * a.es + piece % hc * 16;
            };
            const char* s = place(st + from);
            if (s) {
                x[i] = *(const f32x4*)s;
                to[i] = place(st + j);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (to[i]) *(f32x4*)to[i] = x[i];
}

hipError_t launch_keep(const KeepArgs& a, hipStream_t stream) {
    const int groups = a.Hkv > 0 ? (a.Hkv * (a.D * a.es / 16) + 15) / 16 : 1;
    hipLaunchKernelGGL(k_keep, dim3((unsigned)(a.B * groups), 2), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdr2
