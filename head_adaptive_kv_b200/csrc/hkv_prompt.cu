// hkv_prompt.cu -- the prompt side of the cache: block tables and slot maps
// from request lengths, per-head norms with the position rotation, and the
// tiers filled from pages (C ABI in hkv_prompt.h; the chunk's attention is in
// hkv_chunk.cu).
//
// Every kernel here waits for the kernel before it first of all, and none lets
// its dependent start before it ends: the decode step's kernels read tier
// lengths and queries before their own waits.
#include <cuda_bf16.h>

#include "hkv_device.cuh"
#include "hkv_host.h"
#include "hkv_prompt.h"
#include "hkv_pages.cuh"

namespace hkv {

// =============================================================================
// Page plan and release
//
// One cluster of PLAN_CTAS CTAs. Every CTA scans the requests by itself (a few
// loads a thread; passing the result between CTAs would cost more than the
// scan), the cluster meets once all of them have read the state, and then each
// writes its share of the tables and rows. What bounds it is latency: three
// dependent global loads (lengths, table or stack entry, store) and the scans
// (64 requests of one token: 3.8 us). The release is built the same way: scan,
// a look at its share of the pages for each CTA, meet, and when none has found
// one that is not of the pool, every CTA copies its share back (64 requests of 64
// pages: 3.7 us, of which the look and the second meeting are 1.0).
// =============================================================================

constexpr int PLAN_CTAS = 8;
constexpr int PLAN_NT = 512;

struct PlanP {
    const int32_t *ctx, *fresh, *count_in, *held_in, *stack;
    int32_t *count_out, *held_out, *table, *q_start, *kv_len, *pos, *slot, *granted;
    int64_t table_stride;
    int32_t B, T, page_log2, pages, cols;
    uint32_t *status;
};

__device__ __forceinline__ int cluster_rank()
{
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The word at `local` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_peek(const int *local, int rank)
{
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_addr(local)), "r"(rank)
                 : "memory");
    return v;
}

__global__ void __launch_bounds__(PLAN_NT) k_page_plan(const __grid_constant__ PlanP P)
{
    extern __shared__ __align__(16) int32_t plan_smem[];
    __shared__ unsigned long long red[PLAN_NT / 32];
    // per request: first row, first page (of those given out in this call),
    // cached tokens, pages held before
    int32_t *row0 = plan_smem, *page0 = row0 + P.B + 1, *ctx = page0 + P.B + 1, *held = ctx + P.B;
    wait_prior_grid();
    const int rank = cluster_rank(), tid = threadIdx.x;
    const int mask = (1 << P.page_log2) - 1;
    uint32_t flags = 0;
    int count = __ldcg(P.count_in);
    const int stored_count = count;
    if (count < 0 || count > P.pages) {
        flags |= HKV_DEV_BAD_INDEX;
        count = 0;
    }
    unsigned long long want_pages = 0, want_rows = 0, rows = 0, given = 0;
    for (int b0 = 0; b0 < P.B; b0 += PLAN_NT) {
        const int b = b0 + tid;
        int c = 0, n = 0, h = 0, need = 0;
        bool valid = false;
        if (b < P.B) {
            c = __ldcg(P.ctx + b);
            n = __ldcg(P.fresh + b);
            h = __ldcg(P.held_in + b);
            const int64_t end = (int64_t)c + n;
            valid = c >= 0 && n >= 0 && h >= 0 && h <= P.cols && c <= ((int64_t)h << P.page_log2) &&
                    end <= ((int64_t)P.cols << P.page_log2);
            if (!valid) {
                flags |= HKV_DEV_BAD_INDEX;
                n = 0;
            }
            if (n > 0)
                need = max(0, (int)((end + mask) >> P.page_log2) - h);
        }
        unsigned long long sum_p, sum_r, sum_g;
        const unsigned long long before_p =
            want_pages + block_exclusive_scan<PLAN_NT>((unsigned long long)need, red, &sum_p);
        const unsigned long long before_r =
            want_rows + block_exclusive_scan<PLAN_NT>((unsigned long long)n, red, &sum_r);
        const bool ok = (need == 0 || before_p + need <= (unsigned long long)count) &&
                        (n == 0 || before_r + n <= (unsigned long long)P.T);
        if (!ok)
            flags |= HKV_DEV_PAGES_FULL;
        // rows (at most 2^22) and pages (below 2^27) granted, in one scan
        const unsigned long long grant = ok ? ((unsigned long long)n << 32) | (unsigned)need : 0ull;
        const unsigned long long at = block_exclusive_scan<PLAN_NT>(grant, red, &sum_g);
        if (b < P.B) {
            row0[b] = (int)(rows + (at >> 32));
            page0[b] = (int)(given + (at & 0xffffffffull));
            ctx[b] = c < 0 ? 0 : (int)min((int64_t)c, (int64_t)P.cols << P.page_log2);
            held[b] = h;
        }
        want_pages += sum_p;
        want_rows += sum_r;
        rows += sum_g >> 32;
        given += sum_g & 0xffffffffull;
    }
    if (tid == 0) {
        row0[P.B] = (int)rows;
        page0[P.B] = (int)given;
    }
    __syncthreads();
    cluster_meet();  // every CTA has read the state; it may be overwritten in place

    const int total = (int)rows;
    const int32_t *top = P.stack + count - 1;  // top[-j]: the j-th page given out
    // per request
    for (int b = rank * PLAN_NT + tid; b < P.B; b += PLAN_CTAS * PLAN_NT) {
        const int take = row0[b + 1] - row0[b];
        P.q_start[b] = row0[b];
        P.kv_len[b] = ctx[b] + take;
        P.held_out[b] = held[b] + page0[b + 1] - page0[b];
        if (P.granted)
            P.granted[b] = take;
    }
    if (rank == 0 && tid == 0) {
        P.q_start[P.B] = total;
        *P.count_out = given > 0 ? count - (int)given : stored_count;
    }
    // new columns: a warp per request
    for (int b = rank * (PLAN_NT / 32) + (tid >> 5); b < P.B; b += PLAN_CTAS * (PLAN_NT / 32)) {
        const int j0 = page0[b], got = page0[b + 1] - j0;
        for (int i = tid & 31; i < got; i += 32) {
            const int p = __ldcg(top - (j0 + i));
            if (p < 0 || p >= P.pages)
                flags |= HKV_DEV_BAD_INDEX;
            P.table[b * P.table_stride + held[b] + i] = p;
        }
    }
    // rows: each thread finds its row's request by bisection
    for (int t = rank * PLAN_NT + tid; t < P.T; t += PLAN_CTAS * PLAN_NT) {
        int pos = -1, slot = -1;
        if (t < total) {
            int lo = 0, hi = P.B;  // row0[lo] <= t < row0[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (row0[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            pos = ctx[lo] + t - row0[lo];
            const int col = pos >> P.page_log2, over = col - held[lo];
            const int p = over >= 0 ? __ldcg(top - (page0[lo] + over)) : __ldcg(P.table + lo * P.table_stride + col);
            if (p < 0 || p >= P.pages)
                flags |= HKV_DEV_BAD_INDEX;
            else
                slot = (p << P.page_log2) + (pos & mask);
        }
        P.pos[t] = pos;
        P.slot[t] = slot;
    }
    if (flags)
        atomicOr(P.status, flags);
}

struct ReleaseP {
    const int32_t *done, *count_in, *held_in, *table;
    int32_t *count_out, *held_out, *stack;
    int64_t table_stride;
    int32_t B, pages, cols;
    uint32_t *status;
};

__global__ void __launch_bounds__(PLAN_NT) k_page_release(const __grid_constant__ ReleaseP P)
{
    extern __shared__ __align__(16) int32_t plan_smem[];
    __shared__ unsigned long long red[PLAN_NT / 32];
    __shared__ int found;                           // an entry of this CTA's share is no page of the pool
    int32_t *at = plan_smem, *held = at + P.B + 1;  // first stack entry and pages of each request
    wait_prior_grid();
    const int rank = cluster_rank(), tid = threadIdx.x;
    const int count = __ldcg(P.count_in);
    bool bad = count < 0 || count > P.pages;
    unsigned long long total = 0;
    for (int b0 = 0; b0 < P.B; b0 += PLAN_NT) {
        const int b = b0 + tid;
        int h = 0, back = 0;
        if (b < P.B) {
            h = __ldcg(P.held_in + b);
            if (__ldcg(P.done + b) != 0) {
                bad = bad || h < 0 || h > P.cols;
                back = max(0, min(h, P.cols));
            }
        }
        unsigned long long sum;
        const unsigned long long before = block_exclusive_scan<PLAN_NT>((unsigned long long)back, red, &sum);
        if (b < P.B) {
            // an offset past 32 bits can only be one that is refused below
            at[b] = (int)(total + before);
            held[b] = h;
        }
        total += sum;
    }
    if (tid == 0)
        at[P.B] = (int)total;
    bad = __syncthreads_or(bad || (unsigned long long)max(count, 0) + total > (unsigned long long)P.pages);
    // a warp per request; with `write`, its entries go to the stack, else they are looked at
    const auto entries = [&](bool write) {
        bool wrong = false;
        for (int b = rank * (PLAN_NT / 32) + (tid >> 5); b < P.B; b += PLAN_CTAS * (PLAN_NT / 32)) {
            const int n = at[b + 1] - at[b];
            for (int i = tid & 31; i < n; i += 32) {
                const int p = __ldcg(P.table + b * P.table_stride + i);
                if (write)
                    P.stack[count + at[b] + i] = p;
                else
                    wrong = wrong || p < 0 || p >= P.pages;
            }
        }
        return wrong;
    };
    if (!bad) {
        const bool wrong = __syncthreads_or(entries(false));
        if (tid == 0)
            found = wrong;
    }
    cluster_meet();  // every CTA has read the state and says what it found
    if (!bad)
        bad = __syncthreads_or(tid < PLAN_CTAS && cluster_peek(&found, tid) != 0);
    cluster_meet();  // and has been heard: it may end
    for (int b = rank * PLAN_NT + tid; b < P.B; b += PLAN_CTAS * PLAN_NT)
        P.held_out[b] = !bad && __ldcg(P.done + b) != 0 ? 0 : held[b];
    if (rank == 0 && tid == 0) {
        *P.count_out = bad ? count : count + (int)total;
        if (bad)
            atomicOr(P.status, HKV_DEV_BAD_INDEX);
    }
    if (!bad)
        entries(true);
}

// =============================================================================
// Per-head norm and position rotation
//
// D/8 lanes share a head's row; each holds 8 elements as two chunks of 4,
// chosen so that both elements of every rotated pair sit in one lane: for the
// split form chunks 4l and rot/2 + 4l, for the interleaved form 8l and 8l + 4
// (elements behind rot: 8 in a row). So the rotation needs no exchange, and
// only the sum of squares crosses lanes. A CTA takes TB tokens: its threads
// compute the tokens' cosines and sines once, in 64 bits up to the reduced
// angle, and every head of a token uses them from registers. Reads and writes
// each row once: HBM-bound (16384 tokens, 32 + 2 x 8 heads of 128 in bf16 to
// pages of 64: 80 us, 5.0 TB/s; a CTA's positions, slots and angles stand
// before its first row). Eight tokens: 2.9 us, latency.
// =============================================================================

constexpr int NORM_NT = 256;

struct NormP {
    const char *q, *k, *v;
    int64_t qs, ks, vs;  // byte strides of a token's row
    char *qo, *ko, *vo;  // outputs; ko, vo the pages when slot is given
    int64_t sp, sh, st;  // byte strides of the pages
    const int32_t *pos, *slot;
    const char *qw, *kw;
    const double *inv_freq;
    int32_t T, Hq, Hkv, rot, interleaved, page_log2, pages;
    float eps, mscale;
    uint32_t *status;
};

template <int ES>
struct Chunk4;  // four elements as they lie in memory
template <>
struct Chunk4<2> {
    uint2 w;
    __device__ __forceinline__ void get(float *x) const
    {
        const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
    __device__ __forceinline__ void set(const float *x)
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    __device__ __forceinline__ void load(const char *p) { w = __ldcs(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void store(char *p) const { *reinterpret_cast<uint2 *>(p) = w; }
};
template <>
struct Chunk4<4> {
    float4 w;
    __device__ __forceinline__ void get(float *x) const { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
    __device__ __forceinline__ void set(const float *x) { w = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void load(const char *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void store(char *p) const { *reinterpret_cast<float4 *>(p) = w; }
};

template <int ES, int D, int TB>
__global__ void __launch_bounds__(NORM_NT) k_norm_rope(const __grid_constant__ NormP P)
{
    constexpr int LPR = D / 8;               // lanes of a row
    constexpr int GROUPS = NORM_NT / LPR;    // rows in work at once
    constexpr int GPT = GROUPS / TB;         // of one token
    constexpr int AHEAD = 4;                 // rows a group has in flight
    __shared__ float2 turn[TB][D / 2];       // cosine and sine of each pair
    wait_prior_grid();
    const int t0 = blockIdx.x * TB, half = P.rot / 2;
    for (int i = threadIdx.x; i < TB * half; i += NORM_NT) {
        const int tb = i / half, pair = i - tb * half;
        const int pos = t0 + tb < P.T ? __ldcg(P.pos + t0 + tb) : 0;
        // half turns, reduced to [-1, 1] before the step down to 32 bits
        double x = (double)pos * __ldg(P.inv_freq + pair) * 0.31830988618379067;
        x -= 2.0 * rint(x * 0.5);
        float s, c;
        sincospif((float)x, &s, &c);
        turn[tb][pair] = make_float2(c * P.mscale, s * P.mscale);
    }
    __syncthreads();
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int tb = group % TB, t = t0 + tb;
    if (t >= P.T)
        return;
    const int pos = __ldcg(P.pos + t);
    if (pos < 0)
        return;
    int64_t kv_at = 0;   // where the token's K and V rows go
    bool kv = true;
    int64_t kv_head = (int64_t)D * ES;
    if (P.slot != nullptr) {
        const int slot = __ldcg(P.slot + t);
        const int page = slot >> P.page_log2;
        kv = slot >= 0 && page < P.pages;
        if (!kv && slot != -1 && l == 0 && group / TB == 0)
            atomicOr(P.status, HKV_DEV_BAD_INDEX);
        kv_at = page * P.sp + (slot & ((1 << P.page_log2) - 1)) * P.st;
        kv_head = P.sh;
    } else {
        kv_at = (int64_t)t * P.Hkv * D * ES;
    }
    // this lane's chunks
    const bool paired = P.interleaved ? 8 * l < P.rot : 4 * l < half;
    const int a = P.interleaved ? 8 * l : (paired ? 4 * l : P.rot + 8 * (l - half / 4));
    const int b = P.interleaved || !paired ? a + 4 : half + a;
    float c[4], s[4];
    if (paired) {
        const float4 *src = reinterpret_cast<const float4 *>(&turn[tb][4 * l]);
        const float4 u = src[0], w = src[1];
        c[0] = u.x, s[0] = u.y, c[1] = u.z, s[1] = u.w;
        c[2] = w.x, s[2] = w.y, c[3] = w.z, s[3] = w.w;
    } else {
        for (int i = 0; i < 4; ++i)
            c[i] = 1.0f, s[i] = 0.0f;
    }
    const bool norm = P.qw != nullptr;
    const int H = P.Hq + 2 * P.Hkv;
    const unsigned lanes = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1)));
    Chunk4<ES> wa, wb;
    bool key_weights = false;
    if (norm) {
        wa.load(P.qw + a * ES);
        wb.load(P.qw + b * ES);
    }
    for (int h0 = group / TB; h0 < H; h0 += GPT * AHEAD) {
        Chunk4<ES> xa[AHEAD], xb[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int h = h0 + i * GPT;
            if (h < H) {
                const char *src = h < P.Hq            ? P.q + t * P.qs + (int64_t)h * D * ES
                                  : h < P.Hq + P.Hkv ? P.k + t * P.ks + (int64_t)(h - P.Hq) * D * ES
                                                     : P.v + t * P.vs + (int64_t)(h - P.Hq - P.Hkv) * D * ES;
                xa[i].load(src + a * ES);
                xb[i].load(src + b * ES);
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int h = h0 + i * GPT;
            if (h >= H)
                break;
            const bool is_q = h < P.Hq, is_v = h >= P.Hq + P.Hkv;
            if (!is_q && !kv)
                continue;
            if (!is_v) {
                float x[4], y[4];
                xa[i].get(x);
                xb[i].get(y);
                if (norm) {
                    if (!is_q && !key_weights) {
                        wa.load(P.kw + a * ES);
                        wb.load(P.kw + b * ES);
                        key_weights = true;
                    }
                    float ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(lanes, ss, o);
                    const float r = rsqrtf(ss * (1.0f / D) + P.eps);
                    float u[4], w[4];
                    wa.get(u);
                    wb.get(w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] *= r * u[e];
                        y[e] *= r * w[e];
                    }
                }
                if (paired) {
                    float u[4], w[4];
                    if (P.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            u[e] = x[e] * c[e / 2] - x[e + 1] * s[e / 2];
                            u[e + 1] = x[e + 1] * c[e / 2] + x[e] * s[e / 2];
                            w[e] = y[e] * c[2 + e / 2] - y[e + 1] * s[2 + e / 2];
                            w[e + 1] = y[e + 1] * c[2 + e / 2] + y[e] * s[2 + e / 2];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u[e] = x[e] * c[e] - y[e] * s[e];
                            w[e] = y[e] * c[e] + x[e] * s[e];
                        }
                    }
                    xa[i].set(u);
                    xb[i].set(w);
                } else {
                    xa[i].set(x);
                    xb[i].set(y);
                }
            }
            char *dst = is_q   ? P.qo + ((int64_t)t * P.Hq + h) * D * ES
                        : is_v ? P.vo + kv_at + (h - P.Hq - P.Hkv) * kv_head
                               : P.ko + kv_at + (h - P.Hq) * kv_head;
            xa[i].store(dst + a * ES);
            xb[i].store(dst + b * ES);
        }
    }
}

// =============================================================================
// Tiers from pages
//
// Each CTA moves FILL_TOKENS tokens of one unit, K and V: every thread's loads
// (16 bytes each) are issued before its stores. HBM-bound: rows are read and
// written once (eight prompts of 16384 tokens, 8 heads of 128 in bf16: 155 us,
// 6.5 TB/s). A prompt of 500 tokens: 2.9 us, latency.
// =============================================================================

constexpr int FILL_NT = 256;
constexpr int FILL_TOKENS = 64;

struct FillP {
    PagesP pages;
    const int32_t *kv_len, *take;
    char *dk, *dv, *sk, *sv;
    int64_t dsb, dsh, dst, ssb, ssh, sst;  // byte strides
    int32_t *dlen, *slen, *head, *dropped;
    int32_t Hkv, units, wcap, ncap, blocks;  // blocks: CTAs per unit
    uint32_t *status;
};

template <int ROWB>  // bytes of a row
__global__ void __launch_bounds__(FILL_NT) k_fill_tiers(const __grid_constant__ FillP P)
{
    constexpr int PIECES = ROWB / 16;                       // of a row
    constexpr int PER = 2 * FILL_TOKENS * PIECES / FILL_NT; // pieces a thread moves
    constexpr int BATCH = PER < 8 ? PER : 8;
    wait_prior_grid();
    const int u = blockIdx.x / P.blocks, block = blockIdx.x - u * P.blocks;
    const int b = u / P.Hkv, h = u - b * P.Hkv;
    if (P.take != nullptr && __ldcg(P.take + b) == 0)
        return;
    const int64_t most = (int64_t)P.pages.cols << P.pages.page_log2;
    const int stored = __ldcg(P.kv_len + b);
    const int L = (int)max((int64_t)0, min((int64_t)stored, most));
    const int recent = max(0, L - P.wcap);  // tokens that have left the window
    const int sparse = min(recent, P.ncap);
    if (block == 0 && threadIdx.x == 0) {
        uint32_t flags = 0;
        if (L != stored)
            flags |= HKV_DEV_LEN_CLAMPED;
        if (recent > sparse)
            flags |= HKV_DEV_SPARSE_FULL;
        if (flags)
            atomicOr(P.status, flags);
        if (P.wcap > 0) {
            P.dlen[u] = min(L, P.wcap);
            P.head[u] = recent > 0 ? L % P.wcap : 0;
        }
        if (P.ncap > 0)
            P.slen[u] = sparse;
        if (P.dropped)
            P.dropped[u] = recent - sparse;
    }
    // the tokens kept, dropped ones skipped: kept i is token i below `sparse`, else recent + i - sparse
    const int kept = sparse + L - recent;
    const int i0 = block * FILL_TOKENS;
    if (i0 >= kept)
        return;
    const int64_t dbase = b * P.dsb + h * P.dsh, sbase = b * P.ssb + h * P.ssh;
    bool bad = false;
#pragma unroll
    for (int r0 = 0; r0 < PER; r0 += BATCH) {
        uint4 x[BATCH];
        int tok[BATCH];
#pragma unroll
        for (int r = 0; r < BATCH; ++r) {
            const int piece = (r0 + r) * FILL_NT + threadIdx.x;  // K rows first, then V rows
            const int isv = piece / (FILL_TOKENS * PIECES);
            const int row = piece / PIECES - isv * FILL_TOKENS, off = (piece % PIECES) * 16;
            const int i = i0 + row;
            tok[r] = -1;
            x[r] = make_uint4(0, 0, 0, 0);
            if (i < kept) {
                tok[r] = i < sparse ? i : recent + (i - sparse);
                const int p = page_of(P.pages, b, tok[r]);
                if (p >= 0)
                    x[r] = __ldcs(reinterpret_cast<const uint4 *>((isv ? P.pages.v : P.pages.k) +
                                                                  row_offset(P.pages, p, h, tok[r]) + off));
                else
                    bad = true;
            }
        }
#pragma unroll
        for (int r = 0; r < BATCH; ++r) {
            const int piece = (r0 + r) * FILL_NT + threadIdx.x;
            const int isv = piece / (FILL_TOKENS * PIECES), off = (piece % PIECES) * 16;
            if (tok[r] < 0)
                continue;
            char *dst = tok[r] >= recent
                            ? (isv ? P.dv : P.dk) + dbase + (int64_t)(tok[r] % P.wcap) * P.dst
                            : (isv ? P.sv : P.sk) + sbase + (int64_t)tok[r] * P.sst;
            *reinterpret_cast<uint4 *>(dst + off) = x[r];
        }
    }
    if (bad)
        atomicOr(P.status, HKV_DEV_BAD_INDEX);
}

// =============================================================================
// Host side
// =============================================================================

static hkv_status check_status_ws(const void *ws, size_t ws_bytes)
{
    return ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < 256 ? HKV_ERR_WORKSPACE : HKV_OK;
}

static bool words(const void *p) { return p != nullptr && ptr_aligned(p, 4); }

hkv_status check_pages(const hkv_pages *g, const hkv_problem *p, bool storage, bool table)
{
    if (g == nullptr || g->pages < 0 ||
        (g->page != 16 && g->page != 32 && g->page != 64 && g->page != 128 && g->page != 256) ||
        (int64_t)g->pages * g->page >= (1ll << 31))
        return HKV_ERR_INVALID_ARG;
    if (table && (g->table_cols < 0 || g->table_stride < g->table_cols || (int64_t)g->table_cols * g->page > (1ll << 30) ||
                  (g->table_cols > 0 && !words(g->table))))
        return HKV_ERR_INVALID_ARG;
    if (storage) {
        const int es = es_of(p->dtype);
        if (g->pages > 0 && (g->k == nullptr || g->v == nullptr))
            return HKV_ERR_INVALID_ARG;
        if (!ptr_aligned(g->k, 16) || !ptr_aligned(g->v, 16))
            return HKV_ERR_INVALID_ARG;
        if (g->stride_t < p->D || g->stride_h < 0 || g->stride_p < 0 || (g->stride_t * es) % 16 ||
            (g->stride_h * es) % 16 || (g->stride_p * es) % 16)
            return HKV_ERR_INVALID_ARG;
    }
    return HKV_OK;
}

PagesP pages_p(const hkv_pages *g, int es)
{
    PagesP r{};
    r.k = static_cast<char *>(g->k);
    r.v = static_cast<char *>(g->v);
    r.sp = g->stride_p * es;
    r.sh = g->stride_h * es;
    r.st = g->stride_t * es;
    r.pages = g->pages;
    r.page_log2 = 31 - __builtin_clz((unsigned)g->page);
    r.table = g->table;
    r.table_stride = g->table_stride;
    r.cols = g->table_cols;
    return r;
}

static hkv_status check_states(int32_t B, const hkv_pages *pages, const hkv_page_state *in,
                               const hkv_page_state *after)
{
    if (B < 0 || B > HKV_MAX_REQUESTS || in == nullptr || after == nullptr || in->free != after->free)
        return HKV_ERR_INVALID_ARG;
    const hkv_status s = check_pages(pages, nullptr, false, true);
    if (s != HKV_OK)
        return s;
    if (!words(in->free_count) || !words(after->free_count) || (pages->pages > 0 && !words(in->free)) ||
        (B > 0 && (!words(in->held) || !words(after->held))))
        return HKV_ERR_INVALID_ARG;
    return HKV_OK;
}

}  // namespace hkv

using namespace hkv;

extern "C" {

hkv_status hkv_page_plan(int32_t B, const int32_t *ctx_len, const int32_t *new_len, const hkv_pages *pages,
                         const hkv_page_state *in, const hkv_page_state *after, const hkv_chunk *out,
                         int32_t *granted, void *ws, size_t ws_bytes, hkv_stream_t stream)
{
    hkv_status s = check_states(B, pages, in, after);
    if (s != HKV_OK)
        return s;
    if (out == nullptr || out->tokens < 0 || out->tokens > HKV_MAX_TOKENS || !words(out->q_start) ||
        (out->tokens > 0 && (!words(out->pos) || !words(out->slot))) || !ptr_aligned(granted, 4))
        return HKV_ERR_INVALID_ARG;
    if (B > 0 && (!words(ctx_len) || !words(new_len) || !words(out->kv_len)))
        return HKV_ERR_INVALID_ARG;
    if ((s = check_status_ws(ws, ws_bytes)) != HKV_OK)
        return s;
    PlanP P{};
    P.ctx = ctx_len;
    P.fresh = new_len;
    P.count_in = in->free_count;
    P.held_in = in->held;
    P.stack = in->free;
    P.count_out = after->free_count;
    P.held_out = after->held;
    P.table = pages->table;
    P.table_stride = pages->table_stride;
    P.q_start = out->q_start;
    P.kv_len = out->kv_len;
    P.pos = out->pos;
    P.slot = out->slot;
    P.granted = granted;
    P.B = B;
    P.T = out->tokens;
    P.page_log2 = pages_p(pages, 1).page_log2;
    P.pages = pages->pages;
    P.cols = pages->table_cols;
    P.status = static_cast<uint32_t *>(ws);
    // the shared memory of the most requests: one opt-in for every call
    const size_t smem = (4 * (size_t)B + 2) * sizeof(int32_t);
    int unused = 0;
    if ((s = prepare((const void *)k_page_plan, PLAN_NT, (4 * (size_t)HKV_MAX_REQUESTS + 2) * sizeof(int32_t),
                     &unused)) != HKV_OK)
        return s;
    return launch_dependent(k_page_plan, PLAN_CTAS, PLAN_NT, smem, (cudaStream_t)stream, P, PLAN_CTAS);
}

hkv_status hkv_page_release(int32_t B, const int32_t *done, const hkv_pages *pages, const hkv_page_state *in,
                            const hkv_page_state *after, void *ws, size_t ws_bytes, hkv_stream_t stream)
{
    hkv_status s = check_states(B, pages, in, after);
    if (s != HKV_OK)
        return s;
    if (B > 0 && !words(done))
        return HKV_ERR_INVALID_ARG;
    if ((s = check_status_ws(ws, ws_bytes)) != HKV_OK)
        return s;
    ReleaseP P{};
    P.done = done;
    P.count_in = in->free_count;
    P.held_in = in->held;
    P.table = pages->table;
    P.count_out = after->free_count;
    P.held_out = after->held;
    P.stack = after->free;
    P.table_stride = pages->table_stride;
    P.B = B;
    P.pages = pages->pages;
    P.cols = pages->table_cols;
    P.status = static_cast<uint32_t *>(ws);
    const size_t smem = (2 * (size_t)B + 1) * sizeof(int32_t);
    int unused = 0;
    if ((s = prepare((const void *)k_page_release, PLAN_NT, (2 * (size_t)HKV_MAX_REQUESTS + 1) * sizeof(int32_t),
                     &unused)) != HKV_OK)
        return s;
    return launch_dependent(k_page_release, PLAN_CTAS, PLAN_NT, smem, (cudaStream_t)stream, P, PLAN_CTAS);
}

hkv_status hkv_qk_norm_rope(const hkv_problem *prob, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, int32_t tokens, const int32_t *pos, const int32_t *slot,
                            const hkv_rope *rope, const void *q_w, const void *k_w, float eps, void *q_out,
                            void *k_out, void *v_out, const hkv_pages *pages, void *ws, size_t ws_bytes,
                            hkv_stream_t stream)
{
    hkv_status s = check_problem(prob);
    if (s != HKV_OK)
        return s;
    const int es = es_of(prob->dtype), D = prob->D;
    if (tokens < 0 || tokens > HKV_MAX_TOKENS || rope == nullptr || !(eps >= 0.0f) || (q_w == nullptr) != (k_w == nullptr))
        return HKV_ERR_INVALID_ARG;
    if (rope->rot < 0 || rope->rot > D || (rope->rot > 0 && (rope->inv_freq == nullptr || !ptr_aligned(rope->inv_freq, 8))) ||
        (rope->interleaved != 0 && rope->interleaved != 1) || !(rope->mscale == rope->mscale))
        return HKV_ERR_INVALID_ARG;
    if (rope->rot % 16)
        return HKV_ERR_UNSUPPORTED;
    if (!ptr_aligned(q_w, 16) || !ptr_aligned(k_w, 16))
        return HKV_ERR_INVALID_ARG;
    if (pages != nullptr) {
        if ((s = check_pages(pages, prob, true, false)) != HKV_OK)
            return s;
        if (k_out != nullptr || v_out != nullptr || (tokens > 0 && !words(slot)))
            return HKV_ERR_INVALID_ARG;
    } else if (slot != nullptr || (tokens > 0 && (k_out == nullptr || v_out == nullptr)) || !ptr_aligned(k_out, 16) ||
               !ptr_aligned(v_out, 16)) {
        return HKV_ERR_INVALID_ARG;
    }
    const struct {
        const void *p;
        int64_t stride, heads;
    } rows[3] = {{q, q_stride, prob->Hq}, {k, k_stride, prob->Hkv}, {v, v_stride, prob->Hkv}};
    for (const auto &r : rows)
        if (tokens > 0 && (r.p == nullptr || !ptr_aligned(r.p, 16) || r.stride < r.heads * D || (r.stride * es) % 16))
            return HKV_ERR_INVALID_ARG;
    if (tokens > 0 && (q_out == nullptr || !ptr_aligned(q_out, 16) || !words(pos)))
        return HKV_ERR_INVALID_ARG;
    // A CTA writes its tokens' rows while others still read theirs: an output may stand on its own input row on row,
    // and on nothing else.
    const Span outs[3] = {{q_out, tokens * rows[0].heads * D * es},
                          {k_out, k_out ? tokens * rows[1].heads * D * es : 0},
                          {v_out, v_out ? tokens * rows[2].heads * D * es : 0}};
    for (int o = 0; o < 3 && tokens > 0; ++o) {
        for (int i = 0; i < 3; ++i) {
            const int64_t row = rows[i].heads * D;
            const bool in_place = i == o && outs[o].p == rows[i].p && (tokens == 1 || rows[i].stride == row);
            if (!in_place && outs[o].meets({rows[i].p, ((tokens - 1) * rows[i].stride + row) * es}))
                return HKV_ERR_INVALID_ARG;
        }
        for (int i = 0; i < o; ++i)
            if (outs[o].meets(outs[i]))
                return HKV_ERR_INVALID_ARG;
    }
    if ((s = check_status_ws(ws, ws_bytes)) != HKV_OK)
        return s;
    if (tokens == 0)
        return HKV_OK;
    NormP P{};
    P.q = static_cast<const char *>(q);
    P.k = static_cast<const char *>(k);
    P.v = static_cast<const char *>(v);
    P.qs = q_stride * es;
    P.ks = k_stride * es;
    P.vs = v_stride * es;
    P.qo = static_cast<char *>(q_out);
    P.ko = static_cast<char *>(pages ? pages->k : k_out);
    P.vo = static_cast<char *>(pages ? pages->v : v_out);
    if (pages) {
        const PagesP g = pages_p(pages, es);
        P.sp = g.sp;
        P.sh = g.sh;
        P.st = g.st;
        P.page_log2 = g.page_log2;
        P.pages = g.pages;
        P.slot = slot;
    }
    P.pos = pos;
    P.qw = static_cast<const char *>(q_w);
    P.kw = static_cast<const char *>(k_w);
    P.inv_freq = rope->inv_freq;
    P.T = tokens;
    P.Hq = prob->Hq;
    P.Hkv = prob->Hkv;
    P.rot = rope->rot;
    P.interleaved = rope->interleaved;
    P.eps = eps;
    P.mscale = rope->mscale;
    P.status = static_cast<uint32_t *>(ws);
    const cudaStream_t st = (cudaStream_t)stream;
    // One token a CTA while that leaves some of the 148 SMs free; else eight, whose K and V rows then lie side by side in a page
    // (16384 tokens of 32 + 2 x 8 bf16 heads of 128: 78 us, 81 with four, 84 with 32).
    const int tb = tokens < 4 * 148 ? 1 : 8;
    const int64_t grid = (tokens + tb - 1) / tb;
#define HKV_NORM(E, DD, TT) \
    if (es == E && D == DD && tb == TT) \
        return launch_dependent(k_norm_rope<E, DD, TT>, grid, NORM_NT, 0, st, P);
    HKV_NORM(2, 128, 1) HKV_NORM(2, 128, 8) HKV_NORM(2, 64, 1) HKV_NORM(2, 64, 8)
    HKV_NORM(4, 128, 1) HKV_NORM(4, 128, 8) HKV_NORM(4, 64, 1) HKV_NORM(4, 64, 8)
#undef HKV_NORM
    return HKV_ERR_UNSUPPORTED;
}

hkv_status hkv_fill_tiers(const hkv_problem *prob, const hkv_pages *pages, const int32_t *kv_len,
                          const int32_t *take, const hkv_tier *dense, int32_t *dense_head, const hkv_tier *sparse,
                          int32_t *dropped, void *ws, size_t ws_bytes, hkv_stream_t stream)
{
    hkv_status s = check_problem(prob);
    if (s != HKV_OK)
        return s;
    if ((s = check_tier(dense, prob, true)) != HKV_OK || (s = check_tier(sparse, prob, true)) != HKV_OK ||
        (s = check_pages(pages, prob, true, true)) != HKV_OK)
        return s;
    const int wcap = dense ? dense->cap : 0, ncap = sparse ? sparse->cap : 0;
    if ((wcap > 0 && !words(dense_head)) || !ptr_aligned(dropped, 4) || !ptr_aligned(take, 4) ||
        (prob->B > 0 && !words(kv_len)))
        return HKV_ERR_INVALID_ARG;
    if ((s = check_status_ws(ws, ws_bytes)) != HKV_OK)
        return s;
    const int es = es_of(prob->dtype);
    FillP P{};
    P.pages = pages_p(pages, es);
    P.kv_len = kv_len;
    P.take = take;
    if (wcap > 0) {
        P.dk = static_cast<char *>(const_cast<void *>(dense->k));
        P.dv = static_cast<char *>(const_cast<void *>(dense->v));
        P.dsb = dense->stride_b * es;
        P.dsh = dense->stride_h * es;
        P.dst = dense->stride_t * es;
        P.dlen = const_cast<int32_t *>(dense->len);
        P.head = dense_head;
    }
    if (ncap > 0) {
        P.sk = static_cast<char *>(const_cast<void *>(sparse->k));
        P.sv = static_cast<char *>(const_cast<void *>(sparse->v));
        P.ssb = sparse->stride_b * es;
        P.ssh = sparse->stride_h * es;
        P.sst = sparse->stride_t * es;
        P.slen = const_cast<int32_t *>(sparse->len);
    }
    P.dropped = dropped;
    P.Hkv = prob->Hkv;
    P.units = prob->B * prob->Hkv;
    P.wcap = wcap;
    P.ncap = ncap;
    // as many blocks as the longest request the table and the tiers can hold
    const int64_t most = std::min<int64_t>((int64_t)pages->table_cols * pages->page, (int64_t)wcap + ncap);
    P.blocks = (int32_t)std::max<int64_t>(1, (most + FILL_TOKENS - 1) / FILL_TOKENS);
    P.status = static_cast<uint32_t *>(ws);
    const int64_t grid = (int64_t)P.units * P.blocks;
    if (grid >= (1ll << 31))
        return HKV_ERR_UNSUPPORTED;
    const cudaStream_t st = (cudaStream_t)stream;
    switch (prob->D * es) {
    case 128: return launch_dependent(k_fill_tiers<128>, grid, FILL_NT, 0, st, P);
    case 256: return launch_dependent(k_fill_tiers<256>, grid, FILL_NT, 0, st, P);
    case 512: return launch_dependent(k_fill_tiers<512>, grid, FILL_NT, 0, st, P);
    }
    return HKV_ERR_UNSUPPORTED;
}

}  // extern "C"
