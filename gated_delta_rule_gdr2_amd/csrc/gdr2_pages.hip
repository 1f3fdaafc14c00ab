// Pages for the tokens to come: block tables, slots and packed bounds from request lengths, on gfx950.
//
// Whole numbers, a few hundred KB at most: bound by launches and by the latency of dependent reads. One workgroup
// hands out the pages (running sums over all requests need one order, and a sum of partial results by a second and
// third kernel costs more than it saves at thousands of requests); the slots, which are most of the bytes where
// prompts come in, are written by it too while they are few, and by a second kernel from SLOTS_FEW on.
//
// A request's table entries are read by one thread where it touches at most PAGES_SHORT of them, as every request that goes
// on by a token does, and by a whole wave, 256 entries at a time, where it touches more: those are listed in LDS, and the
// waves take them in turn. Requests of few tokens all of them: each thread writes its own slots.
//
// Measured: 96 requests that go on by a token 3.7 us, 512 of which 24 are prompts of up to 2500 tokens and 16 end 11.3 us
// and 4.4 for the slots.
#include "gdr2_device.hpp"
#include "gdr2_pages.hpp"

namespace gdr2 {

constexpr int PT = 512;           // threads that hand out the pages
// table entries that one thread goes through by itself. Us with 2, 4 and 8, pages of 16 tokens: 2048 requests of one new token
// 10.5, 11.6 and 13.2, of 40 tokens (3 or 4 entries) 161, 20 and 21, of 100 (7 or 8) 162, 163 and 24
constexpr int PAGES_SHORT = 4;
// tokens up to which one workgroup writes the slots: us so and by a second kernel, 96 requests, one of them a prompt of 1500
// tokens 8.7 and 9.5, of 3000 11.7 and 9.7, of 5000 15.7 and 10.4, of 12000 31.4 and 10.1
constexpr int SLOTS_FEW = 2048;

// exclusive prefix sum over the workgroup, and the total; sc: PT / 64 places
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

// Entries first .. end - 1 of a request's table, 256 at a time by a wave: f(index, entry, whether it is a page) for each
// lane's, with f's lanes beyond the end marked by an index of -1. The loads of four steps go out together.
template <class F>
__device__ __forceinline__ void walk_entries(const PagesArgs& a, const int* row, int first, int end, F f) {
    const int l = lane_id();
    for (int i0 = first; i0 < end; i0 += 256) {
        int p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = i0 + 64 * x + l < end ? row[i0 + 64 * x + l] : -1;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (i0 + 64 * x >= end) break;
            const int i = i0 + 64 * x + l;
            f(i < end ? i : -1, p[x], i < end && is_page(a, p[x]));
        }
    }
}

__global__ __launch_bounds__(PT) void k_pages(PagesArgs a) {
    __shared__ long long sc[PT / 64];
    __shared__ int any_gone, any_many, taken, list[PT], number[PT];
    poison_lds((lds_char*)sc, sizeof(sc));
    poison_lds((lds_char*)list, sizeof(list));
    poison_lds((lds_char*)number, sizeof(number));
    poison_lds_done();
    const int tid = threadIdx.x, l = lane_id(), w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const long long cap = (long long)a.max_pages << a.shift;
    const bool direct = a.slots && a.max_tokens <= SLOTS_FEW;  // else a second kernel writes the slots
    const int c0 = tid < a.B ? a.counts[tid] : 0, h0 = tid < a.B ? held_of(a, tid) : 0;
    long long top = a.num_free[0];
    top = top < 0 ? 0 : top < a.pages ? top : a.pages;
    if (tid == 0) any_gone = any_many = taken = 0;
    __syncthreads();
    if (c0 < 0) any_gone = 1;
    if (c0 > PAGES_SHORT) any_many = 1;
    for (int b = tid + PT; b < a.B; b += PT) {
        const int c = a.counts[b];
        if (c < 0) any_gone = 1;
        if (c > PAGES_SHORT) any_many = 1;
    }
    __syncthreads();
    if (any_gone) {
        // ---- requests that end give their pages back, in order
        for (int b0 = 0; b0 < a.B; b0 += PT) {
            const int b = b0 + tid;
            const bool gone = b < a.B && (b0 ? a.counts[b] : c0) < 0;
            long long total;
            const int nth = (int)scan_wg(gone, sc, total);
            if (gone) list[nth] = b;
            __syncthreads();
            const int n = (int)total;
            for (int x = w; x < n; x += PT / 64) {
                int c = 0;
                walk_entries(a, a.table + (size_t)list[x] * a.max_pages, 0, a.max_pages,
                             [&](int, int, bool is) { c += __popcll(__ballot(is)); });
                if (l == 0) number[x] = c;
            }
            __syncthreads();
            const int mine = tid < n ? number[tid] : 0;
            const long long at = scan_wg(mine, sc, total);
            if (tid < n) number[tid] = (int)at;
            __syncthreads();
            for (int x = w; x < n; x += PT / 64) {
                int* row = a.table + (size_t)list[x] * a.max_pages;
                long long p0 = top + number[x];
                walk_entries(a, row, 0, a.max_pages, [&](int i, int p, bool is) {
                    const unsigned long long v = __ballot(is);
                    const long long place = p0 + __popcll(v & ((1ull << l) - 1));
                    if (is && place < a.pages) a.free_pages[place] = p;
                    if (i >= 0) row[i] = -1;
                    p0 += __popcll(v);
                });
            }
            top += total;
            __syncthreads();  // what was given back may be taken below, and the list is free
        }
        if (top > a.pages) top = a.pages;
    }
    // ---- the others take what they lack, in order
    long long tok0 = 0, used = 0;
    for (int b0 = 0; b0 < a.B; b0 += PT) {
        const int b = b0 + tid;
        const bool in = b < a.B;
        const int c = !b0 ? c0 : in ? a.counts[b] : 0, held = !b0 ? h0 : in ? held_of(a, b) : 0, add = c > 0 ? c : 0;
        int* row = a.table + (size_t)(in ? b : 0) * a.max_pages;
        const int lo = held >> a.shift;
        const bool room = add > 0 && held + (long long)add <= cap;
        const int end = room ? (int)((held + (long long)add + a.page - 1) >> a.shift) : lo;
        const bool big = end - lo > PAGES_SHORT;
        int pg[PAGES_SHORT];  // the entries, where they are few
        int n = 0;
#pragma unroll
        for (int i = 0; i < PAGES_SHORT; ++i) {
            pg[i] = !big && lo + i < end ? row[lo + i] : 0;
            n += !big && lo + i < end && !is_page(a, pg[i]);
        }
        long long total;
        const long long tok = tok0 + scan_wg(add, sc, total);
        if (in) a.cu[b] = (int)min(tok, (long long)a.max_tokens);
        tok0 += total;
        const bool fits = room && tok + add <= a.max_tokens;
        int bign = 0, place = 0;
        if (any_many) {  // (more entries than a few need more tokens than a few)
            place = (int)scan_wg(big && fits, sc, total);
            bign = (int)total;
            if (big && fits) list[place] = b;
            __syncthreads();
            for (int x = w; x < bign; x += PT / 64) {
                const int y = list[x], hy = held_of(a, y);
                int k = 0;
                walk_entries(a, a.table + (size_t)y * a.max_pages, hy >> a.shift,
                             (int)(((long long)hy + a.counts[y] + a.page - 1) >> a.shift),
                             [&](int i, int, bool is) { k += __popcll(__ballot(i >= 0 && !is)); });
                if (l == 0) number[x] = k;
            }
            __syncthreads();
            if (big && fits) n = number[place];
        }
        if (!fits) n = 0;
        const long long mine = used + scan_wg(n, sc, total);  // pages taken before
        const bool ok = fits && (n == 0 || mine + n <= top);
        used += total;
        // from the first request on that asks for more than there is, those that lack a page take none: the pages
        // taken are the largest sum that fits
        if (ok && n > 0) atomicMax(&taken, (int)(mine + n));
        if (ok && !big) {
            long long nth = mine;
#pragma unroll
            for (int i = 0; i < PAGES_SHORT; ++i)
                if (lo + i < end && !is_page(a, pg[i])) row[lo + i] = pg[i] = a.free_pages[top - 1 - nth++];
        }
        if (in) a.out[b] = c < 0 ? 0 : ok ? held + add : held;
        if (direct && !any_many)
            for (int j = 0; j < add && tok + j < a.max_tokens; ++j) {
                const int e = ((held + j) >> a.shift) - lo;
                int p = -1;
#pragma unroll
                for (int i = 0; i < PAGES_SHORT; ++i) p = e == i ? pg[i] : p;
                a.slots[tok + j] = ok && is_page(a, p) ? ((long long)p << a.shift) + ((held + j) & (a.page - 1)) : -1;
            }
        if (any_many && bign > 0) {
            if (big && fits) number[place] = ok && n > 0 ? (int)mine : -1;
            __syncthreads();
            for (int x = w; x < bign; x += PT / 64) {
                long long nth = number[x];
                if (nth < 0) continue;
                const int y = list[x], hy = held_of(a, y);
                int* r = a.table + (size_t)y * a.max_pages;
                walk_entries(a, r, hy >> a.shift, (int)(((long long)hy + a.counts[y] + a.page - 1) >> a.shift),
                             [&](int i, int, bool is) {
                                 const bool lack = i >= 0 && !is;
                                 const unsigned long long v = __ballot(lack);
                                 if (lack) r[i] = a.free_pages[top - 1 - (nth + __popcll(v & ((1ull << l) - 1)))];
                                 nth += __popcll(v);
                             });
            }
            __syncthreads();  // the list is free
        }
    }
    __syncthreads();
    const int all = (int)min(tok0, (long long)a.max_tokens);
    if (tid == 0) {
        a.cu[a.B] = all;
        a.num_free[0] = (int)top - taken;
    }
    if (!direct) return;
    if (!any_many) {
        for (int t = all + tid; t < a.max_tokens; t += PT) a.slots[t] = -1;
        return;
    }
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
