// hkv_pages.cuh -- the page pool as the kernels see it, and its host checks.
#pragma once

#include <algorithm>

#include "hkv_prompt.h"

namespace hkv {

struct PagesP {
    char *k, *v;
    int64_t sp, sh, st;  // byte strides of page, KV head, row
    int64_t table_stride;
    const int32_t *table;
    int32_t pages, page_log2, cols;
};

#ifdef __CUDACC__
// Page of request b's token t (0 <= t < cols * page), or -1 when the table
// names none.
__device__ __forceinline__ int page_of(const PagesP &g, int b, int t)
{
    const int p = __ldg(g.table + b * g.table_stride + (t >> g.page_log2));
    return p >= 0 && p < g.pages ? p : -1;
}

// Byte offset of token t's row in page p.
__device__ __forceinline__ int64_t row_offset(const PagesP &g, int p, int h, int t)
{
    return p * g.sp + h * g.sh + (int64_t)(t & ((1 << g.page_log2) - 1)) * g.st;
}
#endif

// storage: K, V and strides are checked against p; table: the block tables.
hkv_status check_pages(const hkv_pages *g, const hkv_problem *p, bool storage, bool table);
PagesP pages_p(const hkv_pages *g, int es);

}  // namespace hkv
