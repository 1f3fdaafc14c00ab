// Pages of a paged key-value cache for the tokens to come: arguments and launcher (internal to libgdr2).
#pragma once
#include <hip/hip_runtime.h>

namespace gdr2 {

struct PagesArgs {
    const int *lengths, *counts;        // [B]
    int *table, *free_pages, *num_free; // [B][max_pages], [pages], [1], updated
    int *out, *cu;                      // [B], [B + 1]
    long long* slots;                   // [max_tokens] or null
    int B, max_tokens, pages, page, shift, max_pages;
};

hipError_t launch_pages(const PagesArgs& a, hipStream_t stream);

}  // namespace gdr2
