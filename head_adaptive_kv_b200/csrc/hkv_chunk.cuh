// hkv_chunk.cuh -- work line, records and merge shared by the kernels of the
// chunk's attention over the paged cache.
//
// Item: M rows (M/G tokens of one request, the G query heads of one KV head
// side by side, so that a K or V row read once serves the whole group). An
// item's keys come in tiles of NK. All items, request by request, head by
// head, stand on one line, ITEM_COST + (its tiles) positions each, C in all,
// and CTA c of N takes the positions [c C / N, (c+1) C / N): equal work for
// every CTA whatever the requests' lengths, one token or many. N is the grid,
// or fewer where that would leave a CTA less than MIN_SHARE positions; the
// rest of the grid has nothing to do. An item that crosses
// from one CTA into the next leaves a record (unnormalised output, row
// maxima and sums) in each, which k_chunk_merge joins in line order; an item
// within one CTA is written at once. A CTA has at most two records: of the
// item it starts in the middle of, and of the one it does not finish.
#pragma once

#include "hkv_device.cuh"
#include "hkv_pages.cuh"

namespace hkv {

constexpr int ITEM_COST = 1;  // line positions of an item beside its tiles
constexpr int MIN_SHARE = 2;  // positions that a CTA is worth (at least 1: an owner of no position has no record)

struct ChunkDesc {  // the item that starts in a CTA and ends in a later one (n > 1 records), or n = 0
    int32_t n, row0, head, rows;  // row0: first token row; rows: valid rows
};

struct ChunkP {
    const char *q;
    int64_t qs;  // byte stride of a token's row
    const int32_t *q_start, *kv_len;
    PagesP pages;
    char *out;
    float *lse;
    float *part;        // records: [2 N][rec_rows][D + 2]
    ChunkDesc *desc;    // [N]
    int32_t B, T, Hq, Hkv, g_log2, rec_rows;
    float scale_log2;   // scale * log2(e)
    uint32_t *status;
    uint64_t wait_ns;
    int32_t withhold;
};

// A request's rows and lengths, clamped to what the buffers hold.
struct ChunkReq {
    int q0, n, kv;
    bool clamped;
};

__device__ __forceinline__ ChunkReq chunk_request(const ChunkP &P, int b)
{
    const int a = __ldg(P.q_start + b), e = __ldg(P.q_start + b + 1), kv = __ldg(P.kv_len + b);
    ChunkReq r;
    r.q0 = max(0, min(a, P.T));
    r.n = max(r.q0, min(e, P.T)) - r.q0;
    r.kv = (int)max((int64_t)0, min((int64_t)kv, (int64_t)P.pages.cols << P.pages.page_log2));
    r.clamped = r.q0 != a || r.q0 + r.n != e || r.kv != kv;
    return r;
}

template <int M, int NK>
struct ChunkLine {
    int tt;  // tokens of an item

    __device__ __forceinline__ explicit ChunkLine(const ChunkP &P) : tt(M >> P.g_log2) {}

    __device__ __forceinline__ int items(const ChunkReq &r) const { return (r.n + tt - 1) / tt; }

    // Tiles of item t on the line: all that its last row may see.
    __device__ __forceinline__ int tiles(const ChunkReq &r, int t) const
    {
        const int ctx = max(0, r.kv - r.n);
        const int full = (ctx + (t + 1) * tt + NK - 1) / NK;
        return t == items(r) - 1 ? min(full, (r.kv + NK - 1) / NK) : full;
    }

    // Line positions of items 0 .. m-1 of one head (m < items): the sum of
    // tiles(t) = floor((a + t tt) / NK), tt a power of two below or above NK.
    __device__ __forceinline__ int64_t before(const ChunkReq &r, int m) const
    {
        const int64_t a = max(0, r.kv - r.n) + tt + NK - 1;
        int64_t s;
        if (tt >= NK) {
            s = m * (a / NK) + (int64_t)(tt / NK) * m * (m - 1) / 2;
        } else {
            // floor((a' + t) / k) with a' = floor(a / tt), k = NK / tt, summed by whole runs of k
            const int64_t k = NK / tt, a1 = a / tt;
            const auto F = [k](int64_t x) {
                const int64_t w = x / k;
                return k * w * (w - 1) / 2 + w * (x - w * k);
            };
            s = F(a1 + m) - F(a1);
        }
        return s + (int64_t)ITEM_COST * m;
    }

    __device__ __forceinline__ int64_t head_cost(const ChunkReq &r) const
    {
        const int m = items(r);
        return m == 0 ? 0 : before(r, m - 1) + ITEM_COST + tiles(r, m - 1);
    }
};

// Where a CTA's share of the line starts and ends.
struct ChunkShare {
    int64_t x0, x1, total;  // positions
    int64_t s;              // start of the first item
    int b, h, t;            // the first item
    int ctas;               // CTAs that share the line
};

// Every thread of the CTA (NT of them) calls this. `red`: NT/32 words.
template <int NT, int M, int NK>
__device__ __forceinline__ void chunk_share(const ChunkP &P, unsigned long long *red, ChunkShare *sh)
{
    const ChunkLine<M, NK> line(P);
    bool clamped = false;
    unsigned long long total = 0;
    for (int b0 = 0; b0 < P.B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        unsigned long long cost = 0;
        if (b < P.B) {
            const ChunkReq r = chunk_request(P, b);
            clamped = clamped || r.clamped;
            cost = (unsigned long long)(line.head_cost(r) * P.Hkv);
        }
        total += block_sum_u64<NT>(cost, red);
    }
    if (clamped && blockIdx.x == 0)
        atomicOr(P.status, HKV_DEV_LEN_CLAMPED);
    const int64_t C = (int64_t)total, N = max((int64_t)1, min((int64_t)gridDim.x, C / MIN_SHARE));
    const bool idle = blockIdx.x >= N;
    const int64_t x0 = idle ? C : C * blockIdx.x / N, x1 = idle ? C : C * (blockIdx.x + 1) / N;
    if (threadIdx.x == 0)
        *sh = ChunkShare{x0, x1, C, 0, P.B, 0, 0, (int)N};
    __syncthreads();
    unsigned long long seen = 0;
    for (int b0 = 0; b0 < P.B && x0 < x1; b0 += NT) {
        const int b = b0 + threadIdx.x;
        unsigned long long cost = 0, sum;
        ChunkReq r{};
        if (b < P.B) {
            r = chunk_request(P, b);
            cost = (unsigned long long)(line.head_cost(r) * P.Hkv);
        }
        const unsigned long long at = seen + block_exclusive_scan<NT>(cost, red, &sum);
        if ((int64_t)at <= x0 && x0 < (int64_t)(at + cost)) {
            const int64_t hc = line.head_cost(r), in = x0 - (int64_t)at;
            const int h = (int)(in / hc);
            const int64_t rest = in - h * hc;
            int lo = 0, hi = line.items(r);  // before(lo) <= rest < before(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (line.before(r, mid) <= rest)
                    lo = mid;
                else
                    hi = mid;
            }
            sh->b = b;
            sh->h = h;
            sh->t = lo;
            sh->s = (int64_t)at + h * hc + line.before(r, lo);
        }
        seen += sum;
        if ((int64_t)seen > x0)
            break;
    }
    __syncthreads();
}

// CTA whose share holds position x.
__device__ __forceinline__ int chunk_owner(const ChunkShare &sh, int64_t x)
{
    return (int)(((x + 1) * sh.ctas - 1) / sh.total);
}

// Walks the items of a CTA's share.
template <int M, int NK>
struct ChunkWalk {
    const ChunkP &P;
    const ChunkLine<M, NK> line;
    const ChunkShare &sh;  // in shared memory
    ChunkReq r;
    int b, h, t, m;
    int64_t s;
    // the present item
    int all;         // its tiles
    int j0, j1;      // this CTA's: [j0, j1)
    int rows, row0;  // valid rows, first token row
    int pos0;        // position of row 0's token
    int limit;       // keys that the last row sees

    __device__ __forceinline__ ChunkWalk(const ChunkP &P_, const ChunkShare &sh_)
        : P(P_), line(P_), sh(sh_), b(sh_.b), h(sh_.h), t(sh_.t), m(0), s(sh_.s)
    {
        if (b < P.B) {
            r = chunk_request(P, b);
            m = line.items(r);
        }
    }

    // The item at the walk's place into the fields above; false at the end.
    __device__ __forceinline__ bool item()
    {
        if (b >= P.B || s >= sh.x1)
            return false;
        const int on_line = line.tiles(r, t), tok = t * line.tt, toks = min(line.tt, r.n - tok);
        rows = toks << P.g_log2;
        row0 = r.q0 + tok;
        pos0 = r.kv - r.n + tok;
        limit = max(0, pos0 + toks);
        all = min(on_line, (limit + NK - 1) / NK);
        const int64_t p = s + ITEM_COST;
        j0 = (int)max((int64_t)0, min((int64_t)all, sh.x0 - p));
        j1 = (int)max((int64_t)0, min((int64_t)all, sh.x1 - p));
        end = p + on_line;
        return true;
    }

    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == all; }
    // An item without tiles belongs to the CTA that holds its first position.
    __device__ __forceinline__ bool mine() const { return all > 0 ? j1 > j0 : s >= sh.x0; }
    __device__ __forceinline__ bool first_part() const { return j0 == 0; }
    __device__ __forceinline__ int parts() const
    {
        const int64_t p = s + ITEM_COST;
        return chunk_owner(sh, p + all - 1) - chunk_owner(sh, p) + 1;
    }

    __device__ __forceinline__ void next()
    {
        s = end;
        if (++t < m)
            return;
        t = 0;
        if (++h < P.Hkv)
            return;
        h = 0;
        do {
            if (++b >= P.B)
                return;
            r = chunk_request(P, b);
            m = line.items(r);
        } while (m == 0);
    }

  private:
    int64_t end;
};

// Joins the records of items that cross CTAs: blocks (c, y) take the item that
// starts in CTA c of the attention's grid, a warp per row. Records are taken
// in line order, so the result does not depend on timing.
constexpr int CMERGE_NT = 256;
constexpr int CMERGE_Y = 4;

template <int ES, int D>
__device__ __forceinline__ void chunk_store(const ChunkP &P, int64_t at, int lane, const float *o, float inv)
{
    constexpr int E = D / 32;
    if constexpr (ES == 4) {
        float *dst = reinterpret_cast<float *>(P.out) + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            dst[e] = o[e] * inv;
    } else {
        uint32_t *dst = reinterpret_cast<uint32_t *>(P.out) + (at * D + lane * E) / 2;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
            dst[e / 2] = *reinterpret_cast<const uint32_t *>(&w);
        }
    }
}

template <int ES, int D>
__global__ void __launch_bounds__(CMERGE_NT) k_chunk_merge(const __grid_constant__ ChunkP P)
{
    constexpr int E = D / 32;
    wait_prior_grid();
    const int c = blockIdx.x / CMERGE_Y;
    const int warp = blockIdx.x % CMERGE_Y * (CMERGE_NT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int4 d = __ldcg(reinterpret_cast<const int4 *>(P.desc) + c);
    const int n = d.x, G = 1 << P.g_log2;
    const int64_t rec = (int64_t)P.rec_rows * (D + 2);
    for (int r = warp; r < (n > 1 ? d.w : 0); r += CMERGE_Y * (CMERGE_NT / 32)) {
        float M = -INFINITY, L = 0.0f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = 0.0f;
        for (int i = 0; i < n; ++i) {
            // the first part is the second record of its CTA, the others are the first of theirs
            const float *at = P.part + (2 * (int64_t)(c + i) + (i == 0 ? 1 : 0)) * rec;
            const float *stats = at + (int64_t)P.rec_rows * D;
            const float mi = __ldcg(stats + r), li = __ldcg(stats + P.rec_rows + r);
            if (mi == -INFINITY)
                continue;
            const float Mn = fmaxf(M, mi), fa = ex2(M - Mn), fb = ex2(mi - Mn);
            L = L * fa + li * fb;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = o[e] * fa + __ldcg(at + (int64_t)r * D + lane * E + e) * fb;
            M = Mn;
        }
        const int64_t at = ((int64_t)d.y + (r >> P.g_log2)) * P.Hq + d.z * G + (r & (G - 1));
        chunk_store<ES, D>(P, at, lane, o, L > 0.0f ? 1.0f / L : 0.0f);
        if (lane == 0 && P.lse != nullptr)
            P.lse[at] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace hkv
