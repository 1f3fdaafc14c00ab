// Pages for the tokens to come: block tables, slots and packed bounds from request lengths, on gfx950.
//
// Whole numbers, a few hundred KB at most: bound by launches and by the latency of dependent reads. One workgroup
// hands out the pages (running sums over all requests need one order, and a sum of partial results by a second and
// third kernel costs more than it saves at thousands of requests); the slots, which are most of the bytes where
// prompts come in, are written by it too while they are few, and by a second kernel from SLOTS_FEW on.
//
// A request's table entries are read by one thread where it touches at most SHORT of them, as every request that goes
// on by a token does, and by a whole wave, one request after another, where it touches more.
#include "gdr2_device.hpp"
#include "gdr2_pages.hpp"

namespace gdr2 {

constexpr int PT = 1024;           // threads that hand out the pages
constexpr int PAGES_SHORT = 4;     // table entries that one thread goes through by itself
constexpr int SLOTS_FEW = 4096;    // tokens up to which one workgroup writes the slots

// exclusive prefix sum over the workgroup, and the total; sc: PT / 64 + 1 places
__device__ __forceinline__ long long scan_wg(long long x, long long* sc, long long& total) {
    const int l = lane_id(), w = threadIdx.x >> 6;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const long long z = __shfl_up(y, o);
        if (l >= o) y += z;
    }
    __syncthreads();  // the last round's sums have been read
    if (l == 63) sc[w] = y;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < PT / 64; ++i) {
        if (i < w) before += sc[i];
        total += sc[i];
    }
    return before + y - x;
}

__device__ __forceinline__ int held_of(const PagesArgs& a, int b) {
    const long long cap = (long long)a.max_pages << a.shift;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n < cap ? n : (int)cap;
}
__device__ __forceinline__ bool is_page(const PagesArgs& a, int p) { return (unsigned)p < (unsigned)a.pages; }

// The place of packed token t, or -1.
__device__ __forceinline__ long long slot_of(const PagesArgs& a, int t) {
    if (t >= a.cu[a.B]) return -1;
    int lo = 0, hi = a.B - 1;  // the last request that begins at or before it
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const int held = held_of(a, lo);
    if (a.out[lo] == held) return -1;  // it got no pages
    const long long pos = (long long)held + (t - a.cu[lo]);
    if ((pos >> a.shift) >= a.max_pages) return -1;
    const int p = a.table[(size_t)lo * a.max_pages + (pos >> a.shift)];
    return is_page(a, p) ? ((long long)p << a.shift) + (pos & (a.page - 1)) : -1;
}

__global__ __launch_bounds__(PT) void k_pages(PagesArgs a) {
    __shared__ long long sc[PT / 64];
    __shared__ int any_gone, taken;
    poison_lds((lds_char*)sc, sizeof(sc));
    poison_lds_done();
    const int tid = threadIdx.x, l = lane_id();
    const long long cap = (long long)a.max_pages << a.shift;
    long long top = a.num_free[0];
    top = top < 0 ? 0 : top < a.pages ? top : a.pages;
    if (tid == 0) any_gone = taken = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += PT)
        if (a.counts[b] < 0) any_gone = 1;
    __syncthreads();
    if (any_gone) {
        // ---- requests that end give their pages back, in order
        for (int b0 = 0; b0 < a.B; b0 += PT) {
            const int b = b0 + tid;
            const bool gone = b < a.B && a.counts[b] < 0;
            const unsigned long long who = __ballot(gone);
            int n = 0;
            for (unsigned long long m = who; m; m &= m - 1) {
                const int x = __builtin_ctzll(m);
                const int* row = a.table + (size_t)(b - l + x) * a.max_pages;
                int c = 0;
                for (int i = l; i < a.max_pages + l; i += 64)
                    c += __popcll(__ballot(i < a.max_pages && is_page(a, row[i < a.max_pages ? i : 0])));
                if (l == x) n = c;
            }
            long long total;
            const long long at = top + scan_wg(n, sc, total);
            for (unsigned long long m = who; m; m &= m - 1) {
                const int x = __builtin_ctzll(m);
                int* row = a.table + (size_t)(b - l + x) * a.max_pages;
                long long p0 = __shfl(at, x);
                for (int i = l; i < a.max_pages + l; i += 64) {
                    const int p = i < a.max_pages ? row[i] : -1;
                    const bool is = i < a.max_pages && is_page(a, p);
                    const unsigned long long v = __ballot(is);
                    const long long place = p0 + __popcll(v & ((1ull << l) - 1));
                    if (is && place < a.pages) a.free_pages[place] = p;
                    if (i < a.max_pages) row[i] = -1;
                    p0 += __popcll(v);
                }
            }
            top += total;
        }
        if (top > a.pages) top = a.pages;
        __syncthreads();  // what was given back may be taken below
    }
    // ---- the others take what they lack, in order
    long long tok0 = 0, used = 0;
    for (int b0 = 0; b0 < a.B; b0 += PT) {
        const int b = b0 + tid;
        const bool in = b < a.B;
        const int c = in ? a.counts[b] : 0, held = in ? held_of(a, b) : 0, add = c > 0 ? c : 0;
        long long total;
        const long long tok = tok0 + scan_wg(add, sc, total);
        if (in) a.cu[b] = (int)min(tok, (long long)a.max_tokens);
        tok0 += total;
        const bool fits = add > 0 && held + (long long)add <= cap && tok + add <= a.max_tokens;
        const int lo = held >> a.shift, hi = fits ? (int)((held + (long long)add + a.page - 1) >> a.shift) : lo;
        const bool big = hi - lo > PAGES_SHORT;
        int* row = a.table + (size_t)(in ? b : 0) * a.max_pages;
        int n = 0;
        if (!big)
            for (int i = lo; i < hi; ++i) n += !is_page(a, row[i]);
        const unsigned long long who = __ballot(big);
        for (unsigned long long m = who; m; m &= m - 1) {
            const int x = __builtin_ctzll(m), i0 = __shfl(lo, x), i1 = __shfl(hi, x);
            const int* r = a.table + (size_t)(b - l + x) * a.max_pages;
            int k = 0;
            for (int i = i0 + l; i < i1 + l; i += 64) k += __popcll(__ballot(i < i1 && !is_page(a, r[i < i1 ? i : i0])));
            if (l == x) n = k;
        }
        const long long mine = used + scan_wg(n, sc, total);  // pages taken before
        const bool ok = fits && (n == 0 || mine + n <= top);
        if (ok && !big) {
            long long nth = mine;
            for (int i = lo; i < hi; ++i)
                if (!is_page(a, row[i])) row[i] = a.free_pages[top - 1 - nth++];
        }
        for (unsigned long long m = __ballot(ok && big && n > 0); m; m &= m - 1) {
            const int x = __builtin_ctzll(m), i0 = __shfl(lo, x), i1 = __shfl(hi, x);
            long long nth = __shfl(mine, x);
            int* r = a.table + (size_t)(b - l + x) * a.max_pages;
            for (int i = i0 + l; i < i1 + l; i += 64) {
                const bool lack = i < i1 && !is_page(a, r[i < i1 ? i : i0]);
                const unsigned long long v = __ballot(lack);
                if (lack) r[i] = a.free_pages[top - 1 - (nth + __popcll(v & ((1ull << l) - 1)))];
                nth += __popcll(v);
            }
        }
        if (in) a.out[b] = c < 0 ? 0 : ok ? held + add : held;
        // from the first request on that asks for more than there is, those that lack a page take none: the pages
        // taken are the largest sum that fits
        if (ok && n > 0) atomicMax(&taken, (int)(mine + n));
        used += total;
    }
    __syncthreads();
    if (tid == 0) {
        a.cu[a.B] = (int)min(tok0, (long long)a.max_tokens);
        a.num_free[0] = (int)top - taken;
    }
    if (!a.slots || a.max_tokens > SLOTS_FEW) return;
    __syncthreads();
    for (int t = tid; t < a.max_tokens; t += PT) a.slots[t] = slot_of(a, t);
}

__global__ __launch_bounds__(256) void k_slots(PagesArgs a) {
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
    if (t < a.max_tokens) a.slots[t] = slot_of(a, (int)t);
}

hipError_t launch_pages(const PagesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(k_pages, dim3(1), dim3(PT), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.slots || a.max_tokens <= SLOTS_FEW) return e;
    hipLaunchKernelGGL(k_slots, dim3((unsigned)((a.max_tokens + 255LL) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdr2
