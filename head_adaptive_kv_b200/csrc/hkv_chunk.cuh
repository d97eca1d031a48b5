// hkv_chunk.cuh -- work line, records and merge shared by the kernels of the
// chunk's attention over the paged cache.
//
// Item: M rows (M/G tokens of one request, the G query heads of one KV head
// side by side, so that a K or V row read once serves the whole group). An
// item's keys come in tiles of NK. All items, request by request, head by
// head, stand on one line, COST + (its tiles) positions each, C in all,
// and CTA c of N takes the positions [c C / N, (c+1) C / N): equal work for
// every CTA whatever the requests' lengths, one token or many. N is the grid,
// or fewer where that would leave a CTA less than LEAST positions; the rest of
// the grid has nothing to do. An item that crosses
// from one CTA into the next leaves a record (unnormalised output, row
// maxima and sums) in each, which k_chunk_merge joins in line order; an item
// within one CTA is written at once. A CTA has at most two records: of the
// item it starts in the middle of, and of the one it does not finish.
#pragma once

#include "hkv_device.cuh"
#include "hkv_pages.cuh"

namespace hkv {

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

__host__ __device__ constexpr int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

// A kernel's line: M rows an item, NK keys a tile, COST positions of an item
// beside its tiles (its beginning and end, in tiles), LEAST positions that a
// CTA is worth (at least 1: an owner of no position has no record). All sizes
// here are powers of two: shifts, as this stands before every call's first load.
template <int M_, int NK_, int COST_, int LEAST_>
struct ChunkLine {
    static constexpr int M = M_, NK = NK_, COST = COST_, LEAST = LEAST_;
    static constexpr int NKL = log2_of(NK);
    int ttl;  // log2 of an item's tokens

    __device__ __forceinline__ explicit ChunkLine(const ChunkP &P) : ttl(log2_of(M) - P.g_log2) {}

    __device__ __forceinline__ int tokens() const { return 1 << ttl; }
    __device__ __forceinline__ int items(const ChunkReq &r) const { return (r.n + tokens() - 1) >> ttl; }

    // Tiles of item t on the line: all that its last row may see.
    __device__ __forceinline__ int tiles(const ChunkReq &r, int t) const
    {
        const int full = (int)((max(0, r.kv - r.n) + ((int64_t)(t + 1) << ttl) + NK - 1) >> NKL);
        return t == items(r) - 1 ? min(full, (int)(((int64_t)r.kv + NK - 1) >> NKL)) : full;
    }

    // Line positions of items 0 .. m-1 of one head (m < items): the sum of
    // tiles(t) = floor((a + (t << ttl)) / NK).
    __device__ __forceinline__ int64_t before(const ChunkReq &r, int m) const
    {
        const int64_t a = (int64_t)max(0, r.kv - r.n) + tokens() + NK - 1;
        int64_t s;
        if (ttl >= NKL) {
            s = m * (a >> NKL) + ((((int64_t)m * (m - 1)) >> 1) << (ttl - NKL));
        } else {
            // floor((a' + t) / k) with a' = floor(a / tokens), k = NK / tokens, summed by whole runs of k
            const int kl = NKL - ttl;
            const int64_t a1 = a >> ttl;
            const auto F = [kl](int64_t x) {
                const int64_t w = x >> kl;
                return (((w * (w - 1)) >> 1) << kl) + w * (x - (w << kl));
            };
            s = F(a1 + m) - F(a1);
        }
        return s + (int64_t)COST * m;
    }

    __device__ __forceinline__ int64_t head_cost(const ChunkReq &r) const
    {
        const int m = items(r);
        return m == 0 ? 0 : before(r, m - 1) + COST + tiles(r, m - 1);
    }
};

// a / b of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ int64_t line_div(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Where a CTA's share of the line starts and ends: C positions over N CTAs,
// C / N each and one more for the first C mod N.
struct ChunkShare {
    int64_t x0, x1;     // positions
    int64_t each, more; // C / N, C mod N
    int64_t s;          // start of the first item
    int b, h, t;        // the first item
    ChunkReq r;         // its request
};

// Every thread of the CTA (NT of them) calls this. `red`: NT/32 words.
template <int NT, class Line>
__device__ __forceinline__ void chunk_share(const ChunkP &P, unsigned long long *red, ChunkShare *sh)
{
    const Line line(P);
    // the cost of request b0 + this thread, the cost of those before it in the strip, and the strip's
    const auto strip = [&](int b0, ChunkReq &r, int64_t &cost, unsigned long long &sum) {
        const int b = b0 + threadIdx.x;
        r = ChunkReq{};
        cost = 0;
        if (b < P.B) {
            r = chunk_request(P, b);
            cost = line.head_cost(r) * P.Hkv;
        }
        return (int64_t)block_exclusive_scan<NT>((unsigned long long)cost, red, &sum);
    };
    ChunkReq r;
    int64_t cost;
    unsigned long long sum;
    int64_t at = strip(0, r, cost, sum), total = (int64_t)sum;
    bool clamped = r.clamped;
    for (int b0 = NT; b0 < P.B; b0 += NT) {
        ChunkReq x;
        int64_t c;
        strip(b0, x, c, sum);
        total += (int64_t)sum;
        clamped = clamped || x.clamped;
    }
    if (clamped && blockIdx.x == 0)
        atomicOr(P.status, HKV_DEV_LEN_CLAMPED);
    const int64_t N = max((int64_t)1, min((int64_t)gridDim.x, line_div(total, Line::LEAST)));
    const int64_t each = line_div(total, N), more = total - each * N, c = blockIdx.x;
    const int64_t x0 = c >= N ? total : c * each + min(c, more), x1 = c >= N ? total : x0 + each + (c < more ? 1 : 0);
    if (threadIdx.x == 0)
        *sh = ChunkShare{x0, x1, each, more, 0, P.B, 0, 0, ChunkReq{}};
    __syncthreads();
    int64_t seen = 0;
    for (int b0 = 0; x0 < x1; b0 += NT) {
        if (b0 > 0)
            at = strip(b0, r, cost, sum);
        else if (P.B > NT)
            at = strip(0, r, cost, sum);
        at += seen;
        if (at <= x0 && x0 < at + cost) {
            const int64_t hc = line.head_cost(r), in = x0 - at;
            const int h = (int)line_div(in, hc);
            const int64_t rest = in - h * hc;
            int lo = 0, hi = line.items(r);  // before(lo) <= rest < before(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (line.before(r, mid) <= rest)
                    lo = mid;
                else
                    hi = mid;
            }
            sh->b = b0 + (int)threadIdx.x;
            sh->h = h;
            sh->t = lo;
            sh->s = at + h * hc + line.before(r, lo);
            sh->r = r;
        }
        seen += (int64_t)sum;
        if (seen > x0 || b0 + NT >= P.B)
            break;
    }
    __syncthreads();
}

// CTA whose share holds position x.
__device__ __forceinline__ int chunk_owner(const ChunkShare &sh, int64_t x)
{
    const int64_t big = sh.more * (sh.each + 1);  // positions of the CTAs with one more
    return (int)(x < big ? line_div(x, sh.each + 1) : sh.more + line_div(x - big, sh.each));
}

// The first request from b on that has rows, or P.B; the lanes of a whole warp
// look at 32 at a time.
__device__ __forceinline__ int chunk_next(const ChunkP &P, int b)
{
#pragma unroll 1
    for (; b < P.B; b += 32) {
        const int x = b + (int)(threadIdx.x & 31);
        const unsigned some = __ballot_sync(0xffffffffu, x < P.B && chunk_request(P, x).n > 0);
        if (some != 0)
            return b + __ffs(some) - 1;
    }
    return P.B;
}

// Walks the items of a CTA's share; whole warps walk together. Idle requests
// behind the share are not looked at, and those within it 32 at a time: with
// steps of one, four requests among 8192 slots took 758 us in bf16; the scan
// of the slots takes 28 to 41.
template <class Line>
struct ChunkWalk {
    const ChunkP &P;
    const Line line;
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
        r = sh.r;
        m = line.items(r);
    }

    // The item at the walk's place into the fields above; false at the end.
    __device__ __forceinline__ bool item()
    {
        if (b >= P.B || s >= sh.x1)
            return false;
        const int on_line = line.tiles(r, t), tok = t << line.ttl, toks = min(line.tokens(), r.n - tok);
        rows = toks << P.g_log2;
        row0 = r.q0 + tok;
        pos0 = r.kv - r.n + tok;
        limit = max(0, pos0 + toks);
        all = min(on_line, (limit + Line::NK - 1) / Line::NK);
        const int64_t p = s + Line::COST;
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
        const int64_t p = s + Line::COST;
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
        if (s >= sh.x1 || ++b >= P.B)  // (item() ends the walk)
            return;
        r = chunk_request(P, b);
        if (r.n == 0) {
            b = chunk_next(P, b + 1);
            if (b >= P.B)
                return;
            r = chunk_request(P, b);
        }
        m = line.items(r);
    }

  private:
    int64_t end;
};

// Joins the records of items that cross CTAs: blocks (c, y) take the item that
// starts in CTA c of the attention's grid, a warp per row, CMERGE_ROWS rows a
// block. Lane i reads the statistics of record i, 32 records at a time; their
// outputs follow four at a time, each four behind the sums of those before: a
// row of n parts takes some n/32 + n/4 round trips to memory, and a warp's two
// rows come one after the other. The order of the sums follows from the number
// of records alone, not from timing. Latency: about 3 us of 16 for one token on
// 2000 keys; few items on a long context are cut into the most parts (one token
// on 32767 keys with one KV head, G 8, bf16: 46 us in all, where its bytes take
// 2.6; 32 tokens behind 16384: 81 us). Joining in the attention's
// kernel instead, by the CTA that finishes an item's last part, takes 1 us off
// there but puts the join behind that CTA's other work: 2048 bf16 tokens alone
// 66 us instead of 59, 16 fp32 tokens on 8000 keys 360 instead of 240.
constexpr int CMERGE_NT = 256;
constexpr int CMERGE_ROWS = 16;

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
    const int blocks = (P.rec_rows + CMERGE_ROWS - 1) / CMERGE_ROWS;
    const int c = blockIdx.x / blocks, r0 = (blockIdx.x - c * blocks) * CMERGE_ROWS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 d = __ldcg(reinterpret_cast<const int4 *>(P.desc) + c);
    const int n = d.x, G = 1 << P.g_log2;
    if (n <= 1)
        return;
    const int64_t rec = (int64_t)P.rec_rows * (D + 2);
    // the first part is the second record of its CTA, the others are the first of theirs
    const auto record = [&](int i) { return P.part + (2 * (int64_t)(c + i) + (i == 0 ? 1 : 0)) * rec; };
    for (int r = r0 + warp; r < min(d.w, r0 + CMERGE_ROWS); r += CMERGE_NT / 32) {
        float M = -INFINITY, L = 0.0f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = 0.0f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            float mi = -INFINITY, li = 0.0f;
            if (i0 + lane < n) {
                const float *stats = record(i0 + lane) + (int64_t)P.rec_rows * D + r;
                mi = __ldcg(stats);
                li = __ldcg(stats + P.rec_rows);
            }
            const float Mn = fmaxf(M, warp_max(mi));
            const float base = Mn == -INFINITY ? 0.0f : Mn;  // no keys so far: all weights 0
            const float f = ex2(M - base), w = ex2(mi - base);
            L = L * f + warp_sum(li * w);
            M = Mn;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] *= f;
            const int some = min(32, n - i0);
#pragma unroll 4
            for (int i = 0; i < some; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i);
                const float *at = record(i0 + i) + (int64_t)r * D + lane * E;
                float x[E];
                if constexpr (E == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(at));
                    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(at));
                    x[0] = v.x, x[1] = v.y;
                }
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[e] = fmaf(x[e], wi, o[e]);
            }
        }
        const int64_t at = ((int64_t)d.y + (r >> P.g_log2)) * P.Hq + d.z * G + (r & (G - 1));
        chunk_store<ES, D>(P, at, lane, o, L > 0.0f ? 1.0f / L : 0.0f);
        if (lane == 0 && P.lse != nullptr)
            P.lse[at] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace hkv
