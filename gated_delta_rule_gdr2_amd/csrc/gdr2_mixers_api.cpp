// C ABI of libgdr2: the gated delta rule with scalar gates, attention over a paged cache and over whole sequences --
// argument validation (host only, before any HIP call), workspace sizing and dispatch. See
// include/gdr2.h for the contract.
#include "../../include/gdr2.h"

#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "gdr2_attn.hpp"
#include "gdr2_kernels.hpp"
#include "gdr2_pages.hpp"
#include "gdr2_prompt.hpp"
#include "gdr2_scalar.hpp"
#include "gdr2_tree.hpp"

namespace {

int esize(int dtype) { return dtype == GDR2_DTYPE_BF16 ? 2 : 4; }

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (p && !aligned(p)) return false;
    return true;
}

// the scalar gates and their gradients are read and written one by one: a whole element is enough
template <size_t N>
bool gates_aligned(const void* const (&ptrs)[N], int esz) {
    for (const void* p : ptrs)
        if ((uintptr_t)p % esz != 0) return false;
    return true;
}

bool sc_supported(int dk, int dv, int dtype) {
    if (dtype == GDR2_DTYPE_BF16) return (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
    return dtype == GDR2_DTYPE_F32 && dk == 64 && dv == 64;
}

// a launch takes fewer than 2^32 threads
bool grid_fits(long long groups, int threads) { return groups < (1LL << 32) / threads; }

// chunk slots: one per chunk, packed also up to one spare per sequence
long long sc_slots(int N, int T, bool packed) {
    return packed ? (long long)T / 64 + N : (long long)N * (((long long)T + 63) / 64);
}

int sc_shape(int N, int T, int Hk, int Hv, int dk, int dv, int dtype, bool packed) {
    if (N < 0 || T < 0 || Hk < 0 || Hv < 0) return GDR2_ERR_SHAPE;
    if (!sc_supported(dk, dv, dtype)) return GDR2_ERR_UNSUPPORTED;
    if (Hk == 0 ? Hv != 0 : Hv == 0 || Hv % Hk != 0) return GDR2_ERR_SHAPE;
    const long long tokens = packed ? T : (long long)N * T;
    // token rows and (sequence, value head, slice)s fit in 32 bits
    if (tokens > 0x7fffffffLL - 64 || (tokens * Hv) > (1LL << 40)) return GDR2_ERR_SHAPE;
    if ((long long)N * Hv * (dv / 16) > 0x7fffffffLL) return GDR2_ERR_SHAPE;
    return GDR2_OK;
}

bool sc_no_tokens(int N, int T, int Hv) { return N == 0 || T == 0 || Hv == 0; }

// ... and for the chunkwise kernels: preparation, gradients and chains (of many walks, two column tiles each)
int sc_chunk_shape(int N, int T, int Hk, int Hv, int dk, int dv, int dtype, bool packed) {
    const int st = sc_shape(N, T, Hk, Hv, dk, dv, dtype, packed);
    if (st != GDR2_OK || sc_no_tokens(N, T, Hv)) return st;
    const long long slots = sc_slots(N, T, packed);
    return grid_fits(slots * Hv, 256) && grid_fits(slots * Hk, 512) &&
                   grid_fits((long long)N * Hv * (dv / 32), gdr2::SC_CHAIN_THREADS)
               ? GDR2_OK : GDR2_ERR_SHAPE;
}

gdr2::ScLayout sc_layout_for(int N, int T, int Hv, int dk, int dv, int dtype, bool packed) {
    int nseg, seglen, lead;
    gdr2::sc_segments(N, T, Hv, dv, packed, nseg, seglen, lead);
    return gdr2::sc_layout(sc_slots(N, T, packed) * Hv, nseg > 1 ? (long long)N * Hv * nseg : 0, dk, dv, esize(dtype));
}

int pass_state(float* dst, const float* src, int N, int Hv, int dk, int dv, void* stream) {
    const long long n = (long long)N * Hv * dk * dv;
    if (!dst || n == 0) return GDR2_OK;
    return gdr2::launch_state_pass(dst, src, n, (hipStream_t)stream) == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

void sc_fill(gdr2::ScArgs& a, const int* cu, int N, int T, int Hk, int Hv, int dk, int dv, int dtype, int zero_rest,
             void* ws) {
    a.cu = cu;
    a.N = N;
    a.T = T;
    a.Hk = Hk;
    a.Hv = Hv;
    a.R = Hv / Hk;
    a.DK = dk;
    a.DV = dv;
    a.slots = (int)sc_slots(N, T, cu != nullptr);
    a.zero_rest = zero_rest;
    gdr2::sc_segments(N, T, Hv, dv, cu != nullptr, a.nseg, a.seglen, a.lead);
    a.L = sc_layout_for(N, T, Hv, dk, dv, dtype, cu != nullptr);
    a.ws = (char*)ws;
}

// A cache's strides: whole 16-byte pieces, so that every row can be read in them; pages of a power of
// two of at least 16 tokens, so that a tile of 16 tokens lies in one page.
int cache_check(const void* k, const void* v, const long long* strides, const int* table, int B, int pages, int page,
                int max_pages, int esz) {
    if (pages < 0 || max_pages < 0) return GDR2_ERR_SHAPE;
    if (page < 16 || page > (1 << 20) || (page & (page - 1)) != 0) return GDR2_ERR_VALUE;
    if (!strides) return GDR2_ERR_NULL;
    for (int i = 0; i < 6; ++i)
        if (strides[i] < 0 || strides[i] % (16 / esz) != 0) return GDR2_ERR_ALIGN;
    if (B > 0 && pages > 0 && max_pages > 0 && (!k || !v || !table)) return GDR2_ERR_NULL;
    return GDR2_OK;
}

void fill_cache(gdr2::Cache& c, const void* k, const void* v, const long long* strides, const int* table, int pages,
                int page, int max_pages) {
    c.k = (void*)k;
    c.v = (void*)v;
    for (int i = 0; i < 3; ++i) {
        c.ks[i] = strides[i];
        c.vs[i] = strides[3 + i];
    }
    c.table = table;
    c.pages = pages;
    c.page = page;
    c.shift = __builtin_ctz(page);
    c.max_pages = max_pages;
}

int attn_shape(int B, int Hq, int Hkv, int D, int dtype) {
    if (B < 0 || Hq < 0 || Hkv < 0) return GDR2_ERR_SHAPE;
    if ((dtype != GDR2_DTYPE_BF16 && dtype != GDR2_DTYPE_F32) || (D != 64 && D != 128)) return GDR2_ERR_UNSUPPORTED;
    if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0) return GDR2_ERR_SHAPE;
    if ((long long)B * Hq > 0x7fffffffLL) return GDR2_ERR_SHAPE;
    return GDR2_OK;
}

// heads of a head group: the matrix cores' 16 columns at most
int group_heads(int Hq, int Hkv) { return Hq / Hkv < 16 ? Hq / Hkv : 16; }

// |scale| log2(e), which masked scores of -inf are multiplied by: a scale of zero weighs all that is seen alike, and so does
// the smallest number above it, times which the largest score is 5e-7, and which leaves -inf what it is.
float scale2_of(float scale) { return fmaxf((float)(fabs((double)scale) * 1.4426950408889634), FLT_TRUE_MIN); }

// Attention over whole sequences: tokens below 2^31 - 1024 (a tile's last row still fits in 32 bits), and launches of
// fewer than 2^32 threads at the smallest tile.
int prompt_shape(int N, int T, int Hq, int Hkv, int D, int dtype, bool packed) {
    if (N < 0 || T < 0) return GDR2_ERR_SHAPE;
    const int st = attn_shape(1, Hq, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    const long long tokens = packed ? T : (long long)N * T;
    if (tokens > 0x7fffffffLL - 1024 || tokens * Hq > (1LL << 40)) return GDR2_ERR_SHAPE;
    if (N > 0 && T > 0 && gdr2::prompt_blocks(N, T, packed) * Hq >= (1LL << 32) / 512) return GDR2_ERR_SHAPE;
    return GDR2_OK;
}
bool prompt_none(int N, int T, int Hq) { return N == 0 || T == 0 || Hq == 0; }

// The backward's workspace: lse2 and delta, fp32 [tokens][Hq] each, then parts of dK and dV, from a multiple of 16 bytes on.
size_t prompt_part_offset(size_t rows) { return (2 * rows * sizeof(float) + 15) / 16 * 16; }

int prompt_fill(gdr2::PromptArgs& a, const long long* strides, const int* cu, int N, int T, int Hq, int Hkv, int D,
                float scale, int window, int dtype, int zero_rest) {
    if (!isfinite(scale) || window < 0) return GDR2_ERR_VALUE;
    const long long heads[3] = {Hq, Hkv, Hkv};
    long long* const to[3] = {a.qs, a.ks, a.vs};
    for (int i = 0; i < 3; ++i) {
        to[i][0] = strides ? strides[2 * i] : heads[i] * D;
        to[i][1] = strides ? strides[2 * i + 1] : D;
        for (int j = 0; j < 2; ++j)
            if (to[i][j] < 0 || to[i][j] % (16 / esize(dtype)) != 0) return GDR2_ERR_ALIGN;
    }
    a.cu = cu;
    a.N = N; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.D = D;
    a.window = window > 0 && window < T ? window : T;
    a.zero_rest = zero_rest;
    a.neg = scale < 0.f;
    a.scale = fabsf(scale);
    a.scale2 = scale2_of(scale);
    return GDR2_OK;
}

int tree_shape(int B, int T, int Hq, int Hkv, int D, int dtype) {
    if (T < 0) return GDR2_ERR_SHAPE;
    const int st = attn_shape(B, Hq, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    if (T > gdr2::TREE_MAX || (long long)B * T * Hq > 0x7fffffffLL) return GDR2_ERR_SHAPE;
    return GDR2_OK;
}

}  // namespace

extern "C" {

size_t gdr2_scalar_workspace_bytes(int N, int T, int Hk, int Hv, int dk, int dv, int packed, int dtype,
                                   int save_for_bwd) {
    if (sc_chunk_shape(N, T, Hk, Hv, dk, dv, dtype, packed != 0) != GDR2_OK || sc_no_tokens(N, T, Hv)) return 0;
    const gdr2::ScLayout L = sc_layout_for(N, T, Hv, dk, dv, dtype, packed != 0);
    return save_for_bwd ? L.train_bytes : L.infer_bytes;
}

int gdr2_scalar_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                    const int* cu_seqlens, void* o, float* ht, int N, int T, int Hk, int Hv, int dk, int dv,
                    int dtype, int zero_rest, int save_for_bwd, void* workspace, size_t workspace_bytes,
                    void* stream) {
    const bool packed = cu_seqlens != nullptr;
    const int st = sc_chunk_shape(N, T, Hk, Hv, dk, dv, dtype, packed);
    if (st != GDR2_OK) return st;
    const bool none = sc_no_tokens(N, T, Hv);
    if (!none && (!q || !k || !v || !g || !beta || !o)) return GDR2_ERR_NULL;
    const void* const ptrs[] = {q, k, v, h0, o, ht, workspace};
    const void* const gates[] = {g, beta};
    if (!all_aligned(ptrs) || !gates_aligned(gates, esize(dtype))) return GDR2_ERR_ALIGN;
    if (none) return pass_state(ht, h0, N, Hv, dk, dv, stream);
    if (!workspace ||
        workspace_bytes < gdr2_scalar_workspace_bytes(N, T, Hk, Hv, dk, dv, packed, dtype, save_for_bwd))
        return GDR2_ERR_WORKSPACE;
    gdr2::ScArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.h0 = h0; a.o = o; a.ht = ht;
    sc_fill(a, cu_seqlens, N, T, Hk, Hv, dk, dv, dtype, zero_rest, workspace);
    return gdr2::launch_sc_fwd(a, dtype == GDR2_DTYPE_BF16, save_for_bwd != 0, (hipStream_t)stream) == hipSuccess
               ? GDR2_OK : GDR2_ERR_HIP;
}

int gdr2_scalar_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                    const void* dout, const float* dht, const int* cu_seqlens, void* dq, void* dk_, void* dv_,
                    void* dg, void* dbeta, float* dh0, int N, int T, int Hk, int Hv, int dk, int dv, int dtype,
                    int zero_rest, int fwd_saved, void* workspace, size_t workspace_bytes, void* stream) {
    const bool packed = cu_seqlens != nullptr;
    const int st = sc_chunk_shape(N, T, Hk, Hv, dk, dv, dtype, packed);
    if (st != GDR2_OK) return st;
    const bool none = sc_no_tokens(N, T, Hv);
    if (!none && (!q || !k || !v || !g || !beta || !dout || !dq || !dk_ || !dv_ || !dg || !dbeta))
        return GDR2_ERR_NULL;
    const void* const ptrs[] = {q, k, v, h0, dout, dht, dq, dk_, dv_, dh0, workspace};
    const void* const gates[] = {g, beta, dg, dbeta};
    if (!all_aligned(ptrs) || !gates_aligned(gates, esize(dtype))) return GDR2_ERR_ALIGN;
    if (none) return pass_state(dh0, dht, N, Hv, dk, dv, stream);
    if (!workspace || workspace_bytes < gdr2_scalar_workspace_bytes(N, T, Hk, Hv, dk, dv, packed, dtype, 1))
        return GDR2_ERR_WORKSPACE;
    gdr2::ScArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.h0 = h0; a.dout = dout; a.dht = dht;
    a.dq = dq; a.dk = dk_; a.dv = dv_; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    sc_fill(a, cu_seqlens, N, T, Hk, Hv, dk, dv, dtype, zero_rest, workspace);
    const bool bf = dtype == GDR2_DTYPE_BF16;
    hipError_t e = hipSuccess;
    if (!fwd_saved) e = gdr2::launch_sc_fwd(a, bf, true, (hipStream_t)stream);
    if (e == hipSuccess) e = gdr2::launch_sc_bwd(a, bf, (hipStream_t)stream);
    return e == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

int gdr2_scalar_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* state,
                     const int* slots, void* o, int B, int T, int Hk, int Hv, int dk, int dv, int n_states, int dtype,
                     void* stream) {
    const int st = sc_shape(B, T, Hk, Hv, dk, dv, dtype, false);
    if (st != GDR2_OK) return st;
    if (n_states < 0 || (!slots && n_states < B)) return GDR2_ERR_SHAPE;
    const bool none = sc_no_tokens(B, T, Hv);
    if (!none && !grid_fits((long long)B * Hv * (dv / 64), 128)) return GDR2_ERR_SHAPE;
    if (!none && (!q || !k || !v || !g || !beta || !o)) return GDR2_ERR_NULL;
    if (!none && n_states > 0 && !state) return GDR2_ERR_NULL;
    const void* const ptrs[] = {q, k, v, state, o};
    const void* const gates[] = {g, beta};
    if (!all_aligned(ptrs) || !gates_aligned(gates, esize(dtype))) return GDR2_ERR_ALIGN;
    if (none) return GDR2_OK;  // no tokens: the states stay as they are
    gdr2::ScStepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.state = state; a.slots = slots; a.o = o;
    a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.R = Hv / Hk; a.states = n_states;
    a.DK = dk; a.DV = dv;
    // as gdr2_step: states of half the Infinity Cache and more go back with non-temporal stores
    a.nt_out = (size_t)B * Hv * dk * dv * sizeof(float) >= (size_t(128) << 20);
    return gdr2::launch_sc_step(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK
                                                                                                 : GDR2_ERR_HIP;
}

size_t gdr2_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int dtype) {
    if (attn_shape(B, Hq, Hkv, D, dtype) != GDR2_OK || B == 0 || Hq == 0) return 0;
    return 2 * (size_t)gdr2::ATTN_WGS * gdr2::attn_part_floats(group_heads(Hq, Hkv), D) * sizeof(float);
}

int gdr2_attn_step(const void* q, const void* k_cache, const void* v_cache, const long long* cache_strides,
                   const int* block_table, const int* lengths, void* o, float* lse, int B, int Hq, int Hkv, int D,
                   int num_pages, int page_size, int max_pages, float scale, int window, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int st = attn_shape(B, Hq, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    if (B == 0 || Hq == 0) return GDR2_OK;
    st = cache_check(k_cache, v_cache, cache_strides, block_table, B, num_pages, page_size, max_pages, esize(dtype));
    if (st != GDR2_OK) return st;
    if (!q || !o || !lengths) return GDR2_ERR_NULL;
    if (!isfinite(scale) || window < 0) return GDR2_ERR_VALUE;
    // token numbers, and the places of all rows' units, fit in 32 bits
    if ((long long)max_pages * page_size > 0x7fffffffLL - 64) return GDR2_ERR_SHAPE;
    gdr2::AttnArgs a = {};
    a.q = q; a.o = o; a.lse = lse; a.lengths = lengths;
    a.part = (float*)workspace;
    // without a page nothing is visible: an empty table says so to the kernels
    fill_cache(a.c, k_cache, v_cache, cache_strides, block_table, num_pages, page_size, num_pages > 0 ? max_pages : 0);
    a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.G = Hq / Hkv;
    a.gh = group_heads(Hq, Hkv);
    a.NG = (a.G + a.gh - 1) / a.gh;
    a.window = window;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    a.wgs = gdr2::ATTN_WGS;
    if (gdr2::attn_line_places(a, gdr2::attn_unit_tokens(dtype == GDR2_DTYPE_BF16)) > 0x7fffffffLL)
        return GDR2_ERR_SHAPE;
    const void* const ptrs[] = {q, k_cache, v_cache, o, workspace};
    if (!all_aligned(ptrs)) return GDR2_ERR_ALIGN;
    if (!workspace || workspace_bytes < gdr2_attn_workspace_bytes(B, Hq, Hkv, D, dtype)) return GDR2_ERR_WORKSPACE;
    return gdr2::launch_attn(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

int gdr2_kv_append(const void* k, const void* v, void* k_cache, void* v_cache, const long long* cache_strides,
                   const int* block_table, const int* starts, const int* cu_seqlens, int B, int tokens, int Hkv, int D,
                   int num_pages, int page_size, int max_pages, int dtype, void* stream) {
    int st = attn_shape(B, Hkv, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    if (tokens < 0 || (!cu_seqlens && tokens != B)) return GDR2_ERR_SHAPE;
    if (B == 0 || tokens == 0 || Hkv == 0) return GDR2_OK;
    if ((long long)tokens * Hkv >= (1LL << 32) / (D / (16 / esize(dtype)))) return GDR2_ERR_SHAPE;  // a thread each
    st = cache_check(k_cache, v_cache, cache_strides, block_table, B, num_pages, page_size, max_pages, esize(dtype));
    if (st != GDR2_OK) return st;
    if (!k || !v || !starts) return GDR2_ERR_NULL;
    const void* const ptrs[] = {k, v, k_cache, v_cache};
    if (!all_aligned(ptrs)) return GDR2_ERR_ALIGN;
    if (num_pages == 0 || max_pages == 0) return GDR2_OK;  // no token has a place
    gdr2::AppendArgs a = {};
    a.k = k; a.v = v; a.starts = starts; a.cu = cu_seqlens;
    fill_cache(a.c, k_cache, v_cache, cache_strides, block_table, num_pages, page_size, max_pages);
    a.B = B; a.tokens = tokens; a.Hkv = Hkv; a.D = D;
    return gdr2::launch_append(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK
                                                                                                : GDR2_ERR_HIP;
}

int gdr2_attn_fwd(const void* q, const void* k, const void* v, const long long* strides, const int* cu_seqlens, void* o,
                  float* lse, void* rest, int N, int T, int Hq, int Hkv, int D, float scale, int window, int dtype,
                  int zero_rest, void* stream) {
    int st = prompt_shape(N, T, Hq, Hkv, D, dtype, cu_seqlens != nullptr);
    if (st != GDR2_OK) return st;
    if (prompt_none(N, T, Hq)) return GDR2_OK;
    if (!q || !k || !v || !o) return GDR2_ERR_NULL;
    gdr2::PromptArgs a = {};
    st = prompt_fill(a, strides, cu_seqlens, N, T, Hq, Hkv, D, scale, window, dtype, zero_rest);
    if (st != GDR2_OK) return st;
    const void* const ptrs[] = {q, k, v, o, rest};
    const void* const floats[] = {lse};
    if (!all_aligned(ptrs) || !gates_aligned(floats, 4)) return GDR2_ERR_ALIGN;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.rest = dtype == GDR2_DTYPE_BF16 ? rest : nullptr;
    return gdr2::launch_prompt_fwd(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK
                                                                                                    : GDR2_ERR_HIP;
}

size_t gdr2_attn_bwd_workspace_bytes(int N, int T, int Hq, int Hkv, int D, int packed, int dtype) {
    if (prompt_shape(N, T, Hq, Hkv, D, dtype, packed != 0) != GDR2_OK || prompt_none(N, T, Hq)) return 0;
    const size_t tokens = (size_t)(packed ? T : (long long)N * T), parts = gdr2::prompt_parts(N, T, Hq, Hkv, packed != 0);
    return parts > 1 ? prompt_part_offset(tokens * Hq) + 2 * parts * tokens * Hkv * D * sizeof(float)
                     : 2 * tokens * Hq * sizeof(float);
}

int gdr2_attn_bwd(const void* q, const void* k, const void* v, const long long* strides, const void* o, const float* lse,
                  const void* rest, const void* dout, const int* cu_seqlens, void* dq, void* dk_, void* dv_, int N, int T,
                  int Hq, int Hkv, int D, float scale, int window, int dtype, int zero_rest, void* workspace,
                  size_t workspace_bytes, void* stream) {
    const bool packed = cu_seqlens != nullptr;
    int st = prompt_shape(N, T, Hq, Hkv, D, dtype, packed);
    if (st != GDR2_OK) return st;
    if (prompt_none(N, T, Hq)) return GDR2_OK;
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk_ || !dv_) return GDR2_ERR_NULL;
    gdr2::PromptArgs a = {};
    st = prompt_fill(a, strides, cu_seqlens, N, T, Hq, Hkv, D, scale, window, dtype, zero_rest);
    if (st != GDR2_OK) return st;
    const void* const ptrs[] = {q, k, v, o, rest, dout, dq, dk_, dv_, workspace};
    const void* const floats[] = {lse};
    if (!all_aligned(ptrs) || !gates_aligned(floats, 4)) return GDR2_ERR_ALIGN;
    if (!workspace || workspace_bytes < gdr2_attn_bwd_workspace_bytes(N, T, Hq, Hkv, D, packed, dtype))
        return GDR2_ERR_WORKSPACE;
    a.q = q; a.k = k; a.v = v; a.o = (void*)o; a.lse = (float*)lse;
    a.rest = dtype == GDR2_DTYPE_BF16 ? (void*)rest : nullptr;
    a.dout = dout; a.dq = dq; a.dk = dk_; a.dv = dv_;
    a.lse2 = (float*)workspace;
    const size_t rows = (size_t)(packed ? T : (long long)N * T) * Hq;
    a.delta = a.lse2 + rows;
    a.part = (float*)((char*)workspace + prompt_part_offset(rows));
    a.parts = gdr2::prompt_parts(N, T, Hq, Hkv, packed);
    return gdr2::launch_prompt_bwd(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK
                                                                                                    : GDR2_ERR_HIP;
}

size_t gdr2_attn_tree_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int dtype) {
    if (tree_shape(B, T, Hq, Hkv, D, dtype) != GDR2_OK || B == 0 || T == 0 || Hq == 0) return 0;
    gdr2::TreeArgs a = {};
    a.T = T; a.G = Hq / Hkv; a.D = D;
    gdr2::tree_rows(a, dtype == GDR2_DTYPE_BF16);
    return gdr2::tree_workspace(a);
}

int gdr2_attn_tree(const void* q, const int* parents, const void* k_cache, const void* v_cache,
                   const long long* cache_strides, const int* block_table, const int* starts, void* o, float* lse, int B,
                   int T, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages, float scale, int window,
                   int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    int st = tree_shape(B, T, Hq, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    if (B == 0 || T == 0 || Hq == 0) return GDR2_OK;
    st = cache_check(k_cache, v_cache, cache_strides, block_table, B, num_pages, page_size, max_pages, esize(dtype));
    if (st != GDR2_OK) return st;
    if (!q || !o || !parents || !starts) return GDR2_ERR_NULL;
    if (!isfinite(scale) || window < 0) return GDR2_ERR_VALUE;
    if ((long long)max_pages * page_size > 0x7fffffffLL - 128) return GDR2_ERR_SHAPE;
    gdr2::TreeArgs a = {};
    a.q = q; a.parents = parents; a.starts = starts; a.o = o; a.lse = lse;
    a.part = (float*)workspace;
    fill_cache(a.c, k_cache, v_cache, cache_strides, block_table, num_pages, page_size, num_pages > 0 ? max_pages : 0);
    a.B = B; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.G = Hq / Hkv;
    a.window = window;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    gdr2::tree_rows(a, dtype == GDR2_DTYPE_BF16);
    a.neg = a.wide && scale < 0.f;
    if (a.wide) a.scale2 = scale2_of(scale);
    if (gdr2::tree_line_places(a) > 0x7fffffffLL) return GDR2_ERR_SHAPE;
    const void* const ptrs[] = {q, k_cache, v_cache, o, workspace};
    const void* const words[] = {parents, starts, block_table, lse};
    if (!all_aligned(ptrs) || !gates_aligned(words, 4)) return GDR2_ERR_ALIGN;
    if (!workspace || workspace_bytes < gdr2_attn_tree_workspace_bytes(B, T, Hq, Hkv, D, dtype)) return GDR2_ERR_WORKSPACE;
    return gdr2::launch_tree(a, dtype == GDR2_DTYPE_BF16, (hipStream_t)stream) == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

int gdr2_kv_keep(void* k_cache, void* v_cache, const long long* cache_strides, const int* block_table, const int* starts,
                 const int* path, int* lengths, int B, int P, int Hkv, int D, int num_pages, int page_size, int max_pages,
                 int dtype, void* stream) {
    int st = attn_shape(B, Hkv, Hkv, D, dtype);
    if (st != GDR2_OK) return st;
    if (P < 0 || P > gdr2::TREE_MAX) return GDR2_ERR_SHAPE;
    if (B == 0) return GDR2_OK;
    st = cache_check(k_cache, v_cache, cache_strides, block_table, B, num_pages, page_size, max_pages, esize(dtype));
    if (st != GDR2_OK) return st;
    if (!starts || (P > 0 && !path)) return GDR2_ERR_NULL;
    const void* const ptrs[] = {k_cache, v_cache};
    const void* const words[] = {block_table, starts, path, lengths};
    if (!all_aligned(ptrs) || !gates_aligned(words, 4)) return GDR2_ERR_ALIGN;
    if ((long long)B * (Hkv * (long long)(D / (16 / esize(dtype))) / 16 + 1) >= (1LL << 32) / 512) return GDR2_ERR_SHAPE;
    gdr2::KeepArgs a = {};
    fill_cache(a.c, k_cache, v_cache, cache_strides, block_table, num_pages, page_size, num_pages > 0 ? max_pages : 0);
    a.starts = starts; a.path = path; a.lengths = lengths;
    a.B = B; a.P = P; a.Hkv = Hkv; a.D = D; a.es = esize(dtype);
    return gdr2::launch_keep(a, (hipStream_t)stream) == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

int gdr2_kv_pages(const int* lengths, const int* counts, int* block_table, int* free_pages, int* num_free,
                  int* new_lengths, int* cu_seqlens, long long* slots, int B, int max_tokens, int num_pages, int page_size,
                  int max_pages, void* stream) {
    if (B < 0 || max_tokens < 0 || num_pages < 0 || max_pages < 0) return GDR2_ERR_SHAPE;
    if (page_size < 16 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0) return GDR2_ERR_VALUE;
    if ((long long)max_pages * page_size > 0x7fffffffLL) return GDR2_ERR_SHAPE;
    if (!num_free || !cu_seqlens) return GDR2_ERR_NULL;
    if (B > 0 && (!lengths || !counts || !new_lengths || (max_pages > 0 && !block_table))) return GDR2_ERR_NULL;
    if (num_pages > 0 && !free_pages) return GDR2_ERR_NULL;
    const void* const words[] = {lengths, counts, block_table, free_pages, num_free, new_lengths, cu_seqlens};
    const void* const longs[] = {slots};
    if (!gates_aligned(words, 4) || !gates_aligned(longs, 8)) return GDR2_ERR_ALIGN;
    gdr2::PagesArgs a = {};
    a.lengths = lengths; a.counts = counts; a.table = block_table; a.free_pages = free_pages; a.num_free = num_free;
    a.out = new_lengths; a.cu = cu_seqlens; a.slots = max_tokens > 0 ? slots : nullptr;
    a.B = B; a.max_tokens = max_tokens; a.pages = num_pages; a.page = page_size;
    a.shift = __builtin_ctz(page_size);
    a.max_pages = max_pages;
    return gdr2::launch_pages(a, (hipStream_t)stream) == hipSuccess ? GDR2_OK : GDR2_ERR_HIP;
}

}  // extern "C"
