// hkv_chunk.cu -- attention of a chunk of new tokens over the paged cache
// (C ABI in hkv_prompt.h). The work line and the merge are in hkv_chunk.cuh.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "hkv_chunk.cuh"
#include "hkv_chunk_mma.cuh"
#include "hkv_host.h"

namespace hkv {

// =============================================================================
// 32-bit kernel: fp32 products on the FMA units
//
// 16 x 16 threads; thread (y, x) holds rows y + 16 i and, of a tile's 64 keys,
// x + 16 j; of the output columns 4 x + 64 c. K and V tiles land by cp.async;
// the weights take K's place in shared memory once the scores are formed, and
// two CTAs an SM cover each other's waits. Bound by FMAs and the reads of
// shared memory that feed them: a thread's 4 x 4 scores take 8 reads of 16
// bytes for 64 FMAs (2048 tokens behind 2048, Hq 8, Hkv 2, D 128: 657 us, 39
// TFLOP/s).
// =============================================================================

constexpr int FC_NT = 256;
constexpr int FC_NK = 64;
constexpr int FC_M = 64;
using FcLine = ChunkLine<FC_M, FC_NK, 1, 1>;

template <int D>
struct FcSmem {
    float q[FC_M][D + 4];
    float k[FC_NK][D + 4];  // then the weights, [FC_M][FC_NK + 4]
    float v[FC_NK][D];
    ChunkShare share;
    unsigned long long red[FC_NT / 32];
    int ok[FC_NK];  // the tile's keys that are there
};

template <int D>
__global__ void __launch_bounds__(FC_NT, 2) k_chunk_fma(const __grid_constant__ ChunkP P)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<FcSmem<D> *>(smem_raw);
    constexpr int M = FC_M, RT = M / 16, CT = D / 64;
    static_assert(M * (FC_NK + 4) <= FC_NK * (D + 4), "the weights fit in K's place");
    float(*w)[FC_NK + 4] = reinterpret_cast<float(*)[FC_NK + 4]>(&sm.k[0][0]);
    wait_prior_grid();
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    if (tid == 0)
        P.desc[blockIdx.x].n = 0;
    chunk_share<FC_NT, FcLine>(P, sm.red, &sm.share);
    const int G = 1 << P.g_log2;
    const int64_t rec = (int64_t)P.rec_rows * (D + 2);
    bool bad = false;
    for (ChunkWalk<FcLine> it(P, sm.share); it.item(); it.next()) {
        if (!it.mine())
            continue;
        cp_async_wait_all();
        __syncthreads();  // the item before is done with q
        for (int i = tid; i < M * (D / 4); i += FC_NT) {
            const int r = i / (D / 4), x = i % (D / 4);
            if (r < it.rows)
                cp_async16(&sm.q[r][4 * x], P.q + (it.row0 + (r >> P.g_log2)) * P.qs +
                                                ((int64_t)(it.h * G + (r & (G - 1))) * D + 4 * x) * 4);
            else
                *reinterpret_cast<float4 *>(&sm.q[r][4 * x]) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mx[RT], sum[RT];
        float4 o[RT][CT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            mx[i] = -INFINITY;
            sum[i] = 0.0f;
#pragma unroll
            for (int c = 0; c < CT; ++c)
                o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int j = it.j0; j < it.j1; ++j) {
            const int key0 = j * FC_NK;
            __syncthreads();  // the tile before is done with k, v and ok
            for (int i = tid; i < FC_NK * (D / 4); i += FC_NT) {
                const int r = i / (D / 4), x = i % (D / 4), key = key0 + r;
                const int p = key < it.r.kv ? page_of(P.pages, it.b, key) : -1;
                if (x == 0) {
                    sm.ok[r] = p >= 0;
                    bad = bad || (p < 0 && key < it.r.kv);
                }
                if (p >= 0) {
                    const int64_t at = row_offset(P.pages, p, it.h, key) + 16 * x;
                    cp_async16(&sm.k[r][4 * x], P.pages.k + at);
                    cp_async16(&sm.v[r][4 * x], P.pages.v + at);
                } else {
                    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4 *>(&sm.k[r][4 * x]) = none;
                    *reinterpret_cast<float4 *>(&sm.v[r][4 * x]) = none;
                }
            }
            cp_async_wait_all();  // (the queries', too, before the first tile)
            __syncthreads();
            float2 s2[RT][4];  // even and odd elements, two products an instruction
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    s2[i][n] = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 a[RT], b[4];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    a[i] = lds4(&sm.q[ty + 16 * i][d]);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    b[n] = lds4(&sm.k[tx + 16 * n][d]);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        s2[i][n] = ffma2(make_float2(a[i].x, a[i].y), make_float2(b[n].x, b[n].y), s2[i][n]);
                        s2[i][n] = ffma2(make_float2(a[i].z, a[i].w), make_float2(b[n].z, b[n].w), s2[i][n]);
                    }
            }
            float s[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    s[i][n] = s2[i][n].x + s2[i][n].y;
            int ok[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                ok[n] = sm.ok[tx + 16 * n];
            __syncthreads();  // k has been read: the weights take its place
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int pos = it.pos0 + ((ty + 16 * i) >> P.g_log2);
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const bool on = ok[n] && key0 + tx + 16 * n <= pos;
                    s[i][n] = on ? s[i][n] * P.scale_log2 : -INFINITY;
                    top = fmaxf(top, s[i][n]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float mn = fmaxf(mx[i], top);
                const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing yet: all weights 0
                const float f = ex2(mx[i] - ref);
                mx[i] = mn;
                sum[i] *= f;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    o[i][c].x *= f;
                    o[i][c].y *= f;
                    o[i][c].z *= f;
                    o[i][c].w *= f;
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float p = ex2(s[i][n] - ref);
                    sum[i] += p;
                    w[ty + 16 * i][tx + 16 * n] = p;
                }
            }
            __syncthreads();
#pragma unroll 4
            for (int n = 0; n < FC_NK; n += 4) {
                float4 p[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    p[i] = lds4(&w[ty + 16 * i][n]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const float4 v = lds4(&sm.v[n + e][4 * tx + 64 * c]);
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                            const float2 pp = make_float2(pe, pe);
                            const float2 u = ffma2(pp, make_float2(v.x, v.y), make_float2(o[i][c].x, o[i][c].y));
                            const float2 w2 = ffma2(pp, make_float2(v.z, v.w), make_float2(o[i][c].z, o[i][c].w));
                            o[i][c] = make_float4(u.x, u.y, w2.x, w2.y);
                        }
                    }
            }
        }
        const bool whole = it.whole();
        float *record = P.part + (2 * (int64_t)blockIdx.x + (it.first_part() ? 1 : 0)) * rec;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty + 16 * i;
            float l = sum[i];
#pragma unroll
            for (int x = 8; x > 0; x >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, x);
            if (r >= it.rows)
                continue;
            const float inv = whole ? (l > 0.0f ? 1.0f / l : 0.0f) : 1.0f;
            const int64_t at = (int64_t)(it.row0 + (r >> P.g_log2)) * P.Hq + it.h * G + (r & (G - 1));
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float4 v =
                    make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv);
                const int col = 4 * tx + 64 * c;
                if (!whole) {
                    float2 *dst = reinterpret_cast<float2 *>(record + (int64_t)r * D + col);
                    dst[0] = make_float2(v.x, v.y);
                    dst[1] = make_float2(v.z, v.w);
                } else {
                    *reinterpret_cast<float4 *>(P.out + (at * D + col) * 4) = v;
                }
            }
            if (tx == 0) {
                if (!whole) {
                    record[(int64_t)P.rec_rows * D + r] = mx[i];
                    record[(int64_t)P.rec_rows * (D + 1) + r] = l;
                } else if (P.lse != nullptr) {
                    P.lse[at] = l > 0.0f ? (mx[i] + log2f(l)) * 0.6931471805599453f : -INFINITY;
                }
            }
        }
        if (tid == 0 && !whole && it.first_part())
            P.desc[blockIdx.x] = ChunkDesc{it.parts(), it.row0, it.h, it.rows};
    }
    cp_async_wait_all();
    if (bad)
        atomicOr(P.status, HKV_DEV_BAD_INDEX);
}

// =============================================================================
// 32-bit kernel for single tokens
//
// An item is one token's G rows of a KV head. Each warp takes key groups of
// its own (every FR_WARPS-th of 32 keys) and keeps a maximum, sum and output
// for each row; the warps meet at the item's end. Scores: four keys at a time,
// 8 lanes a key, each lane D/8 elements against its part of the G queries in
// registers (two keys and 16 lanes at G = 8). Output: a lane holds D/32
// columns, V rows are read whole by the warp. K and V go from memory to
// registers and are used once for all G rows, 8 x G FMAs a lane for 16 bytes
// each: bound by loads in flight (16 tokens on 8000 keys each, Hq 32, Hkv 8,
// D 128: 240 us, 4.4 TB/s).
// =============================================================================

constexpr int FR_WARPS = 4;
constexpr int FR_NK = 32 * FR_WARPS;  // keys of a tile: one group a warp

template <int D, int G>
struct FrSmem {
    ChunkShare share;
    unsigned long long red[FR_WARPS];
    float m[FR_WARPS][G], l[FR_WARPS][G], o[FR_WARPS][G][D];
};

template <int D, int G>
__global__ void __launch_bounds__(FR_WARPS * 32, 4) k_chunk_rows(const __grid_constant__ ChunkP P)
{
    // lanes of a key: a lane's part of the queries is at most 64 registers (at D 128, 616 bytes spill at G 8 all the
    // same, and 72 at G 4)
    constexpr int LK = G == 8 ? 16 : 8;
    using Line = ChunkLine<G, FR_NK, 1, 1>;
    constexpr int KS = 32 / LK;            // keys at a time
    constexpr int E = D / LK, C = D / 32;  // elements of a key a lane, output columns a lane
    __shared__ FrSmem<D, G> sm;
    wait_prior_grid();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LK, kq = lane / LK;
    if (threadIdx.x == 0)
        P.desc[blockIdx.x].n = 0;
    chunk_share<FR_WARPS * 32, Line>(P, sm.red, &sm.share);
    const int64_t rec = (int64_t)P.rec_rows * (D + 2);
    bool bad = false;
    for (ChunkWalk<Line> it(P, sm.share); it.item(); it.next()) {
        if (!it.mine())
            continue;
        float q[G][E];
        const char *qrow = P.q + it.row0 * P.qs + (int64_t)it.h * G * D * 4;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(qrow + (g * D + LK * i + 4 * sub) * 4));
                q[g][i] = x.x, q[g][i + 1] = x.y, q[g][i + 2] = x.z, q[g][i + 3] = x.w;
            }
        float m[G], l[G], o[G][C];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                o[g][c] = 0.0f;
        }
        for (int j = it.j0; j < it.j1; ++j) {
            const int key0 = j * FR_NK + warp * 32, n = min(32, it.limit - key0);
            if (n <= 0)
                continue;
            // lane i: key key0 + i's row, or -1
            int64_t at = -1;
            if (lane < n) {
                const int p = page_of(P.pages, it.b, key0 + lane);
                bad = bad || p < 0;
                if (p >= 0)
                    at = row_offset(P.pages, p, it.h, key0 + lane);
            }
            float s[G];  // lane i: the scores of key key0 + i
#pragma unroll
            for (int g = 0; g < G; ++g)
                s[g] = -INFINITY;
#pragma unroll 2
            for (int k = 0; k < 32; k += KS) {
                if (k >= n)
                    break;
                const int64_t row = __shfl_sync(0xffffffffu, at, k + kq);
                float x[E];
#pragma unroll
                for (int i = 0; i < E; i += 4) {
                    const float4 v = row < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                             : __ldg(reinterpret_cast<const float4 *>(P.pages.k + row + (LK * i + 4 * sub) * 4));
                    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float d = 0.0f;
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        d = fmaf(q[g][i], x[i], d);
#pragma unroll
                    for (int i = 1; i < LK; i *= 2)
                        d += __shfl_xor_sync(0xffffffffu, d, i);
                    // key k + i is with the lanes LK i ..
                    const float mine = __shfl_sync(0xffffffffu, d, LK * (lane % KS));
                    if (lane / KS == k / KS)
                        s[g] = mine;
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                s[g] = at < 0 ? -INFINITY : s[g] * P.scale_log2;
                const float mn = fmaxf(m[g], warp_max(s[g]));
                const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing yet: all weights 0
                const float f = ex2(m[g] - ref);
                s[g] = ex2(s[g] - ref);
                m[g] = mn;
                l[g] = l[g] * f + s[g];  // this lane's keys; summed over the lanes at the end
#pragma unroll
                for (int c = 0; c < C; ++c)
                    o[g][c] *= f;
            }
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const int64_t row = __shfl_sync(0xffffffffu, at, k);
                float v[C];
#pragma unroll
                for (int c = 0; c < C; ++c)
                    v[c] = 0.0f;
                if (row >= 0) {
                    const char *src = P.pages.v + row + lane * C * 4;
                    if constexpr (C == 4) {
                        const float4 x = __ldg(reinterpret_cast<const float4 *>(src));
                        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                    } else {
                        const float2 x = __ldg(reinterpret_cast<const float2 *>(src));
                        v[0] = x.x, v[1] = x.y;
                    }
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float p = __shfl_sync(0xffffffffu, s[g], k);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        o[g][c] = fmaf(p, v[c], o[g][c]);
                }
            }
        }
        // the warps' parts together, in warp order
        __syncthreads();  // the item before has been read
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float sum = warp_sum(l[g]);
            if (lane == 0) {
                sm.m[warp][g] = m[g];
                sm.l[warp][g] = sum;
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                sm.o[warp][g][lane * C + c] = o[g][c];
        }
        __syncthreads();
        const bool whole = it.whole();
        float *record = P.part + (2 * (int64_t)blockIdx.x + (it.first_part() ? 1 : 0)) * rec;
        for (int i = threadIdx.x; i < G * D; i += FR_WARPS * 32) {
            const int g = i / D, d = i - g * D;
            float M = -INFINITY, L = 0.0f, x = 0.0f;
#pragma unroll
            for (int w = 0; w < FR_WARPS; ++w)
                M = fmaxf(M, sm.m[w][g]);
            const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int w = 0; w < FR_WARPS; ++w) {
                const float f = ex2(sm.m[w][g] - ref);
                L = fmaf(sm.l[w][g], f, L);
                x = fmaf(sm.o[w][g][d], f, x);
            }
            const int64_t at = (int64_t)it.row0 * P.Hq + it.h * G + g;
            if (whole) {
                reinterpret_cast<float *>(P.out)[at * D + d] = L > 0.0f ? x / L : 0.0f;
                if (d == 0 && P.lse != nullptr)
                    P.lse[at] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
            } else {
                record[(int64_t)g * D + d] = x;
                if (d == 0) {
                    record[(int64_t)P.rec_rows * D + g] = M;
                    record[(int64_t)P.rec_rows * (D + 1) + g] = L;
                }
            }
        }
        if (threadIdx.x == 0 && !whole && it.first_part())
            P.desc[blockIdx.x] = ChunkDesc{it.parts(), it.row0, it.h, it.rows};
    }
    if (bad)
        atomicOr(P.status, HKV_DEV_BAD_INDEX);
}

// =============================================================================
// Host side
// =============================================================================

struct ChunkWs {
    size_t desc, part, total;
    int rec_rows, ctas;
};

static ChunkWs chunk_ws(const hkv_problem *p, int32_t tokens)
{
    ChunkWs w{};
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const bool bf = p->dtype == HKV_BF16;
    w.ctas = bf ? sms : 4 * sms;  // fp32: single tokens in CTAs of half the threads
    const int64_t rows = std::min<int64_t>(bf ? CM_M : FC_M, (int64_t)tokens * (p->Hq / p->Hkv));
    w.rec_rows = (int)((rows + 7) / 8 * 8);
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.desc = 256;
    w.part = w.desc + up((size_t)w.ctas * sizeof(ChunkDesc));
    w.total = w.part + up((size_t)2 * w.ctas * w.rec_rows * (p->D + 2) * 4);
    return w;
}

static int64_t merge_blocks(const ChunkP &P, int ctas)
{
    return (int64_t)ctas * ((P.rec_rows + CMERGE_ROWS - 1) / CMERGE_ROWS);
}

// Tiled maps of the bf16 kernel, boxes of 64 elements (128 bytes, swizzled) by
// 128 rows: q as [T][Hq][D] in boxes of one KV head's group, K and V as
// [pages][Hkv][page][D] in boxes of a page (half a page of 256).
static bool encode_box(CUtensorMap *m, const void *base, int dims, const cuuint64_t *dim, const cuuint64_t *stride,
                       const cuuint32_t *box)
{
    const auto enc = tensor_map_encoder();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc != nullptr &&
           enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(base), dim, stride, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static hkv_status encode_maps(const hkv_problem *p, const ChunkP &A, ChunkMmaP *M)
{
    const cuuint64_t D = (cuuint64_t)p->D;
    const cuuint32_t G = (cuuint32_t)(p->Hq / p->Hkv);
    const cuuint64_t qd[3] = {D, (cuuint64_t)p->Hq, (cuuint64_t)A.T}, qst[2] = {D * 2, (cuuint64_t)A.qs};
    const cuuint32_t qb[3] = {64, G, 128 / G}, qb1[3] = {64, G, 1};
    const PagesP &g = A.pages;
    const cuuint64_t page = 1ull << g.page_log2, pages = (cuuint64_t)std::max(g.pages, 1);
    const cuuint64_t kd[4] = {D, page, (cuuint64_t)p->Hkv, pages};
    // the stride of a dimension of one is never used, but has to be valid
    const cuuint64_t row = (cuuint64_t)g.st, head = p->Hkv > 1 ? (cuuint64_t)g.sh : row;
    const cuuint64_t kst[3] = {row, head, g.pages > 1 ? (cuuint64_t)g.sp : row};
    const cuuint32_t kb[4] = {64, (cuuint32_t)std::min<cuuint64_t>(page, CM_NK), 1, 1};
    // an empty pool has no address: no load reads through its maps
    const void *k = g.pages > 0 ? (const void *)g.k : (const void *)A.q;
    const void *v = g.pages > 0 ? (const void *)g.v : (const void *)A.q;
    M->none = (int32_t)pages;
    return encode_box(&M->q, A.q, 3, qd, qst, qb) && encode_box(&M->q1, A.q, 3, qd, qst, qb1) &&
                   encode_box(&M->k, k, 4, kd, kst, kb) && encode_box(&M->v, v, 4, kd, kst, kb)
               ? HKV_OK
               : HKV_ERR_INVALID_ARG;
}

template <int D>
static hkv_status run_mma(const hkv_problem *p, const ChunkP &A, int ctas, cudaStream_t st)
{
    ChunkMmaP M{};
    M.c = A;
    hkv_status s = encode_maps(p, A, &M);
    if (s != HKV_OK)
        return s;
    if ((s = launch_dependent(k_chunk_mma<D>, ctas, CM_NT, sizeof(CmSmem<D>) + 1024, st, M)) != HKV_OK)
        return s;
    return launch_dependent(k_chunk_merge<2, D>, merge_blocks(A, ctas), CMERGE_NT, 0, st, A);
}

template <int D>
static hkv_status run_fma(const ChunkP &P, int ctas, cudaStream_t st)
{
    hkv_status s;
    // No more rows than requests: single tokens, as far as the host can tell. Any lengths are right in either kernel,
    // but not as fast: 16 single tokens on 8000 keys (Hq 32, Hkv 8, D 128) take 240 us here and 858 in the kernel for
    // chunks, where a batch with room for more rows than requests goes; 48 tokens of one request behind 8000 keys, in a
    // table of 64, take 425 us here and 180 there.
    if (P.T <= P.B) {
        const auto rows = P.g_log2 == 0   ? k_chunk_rows<D, 1>
                          : P.g_log2 == 1 ? k_chunk_rows<D, 2>
                          : P.g_log2 == 2 ? k_chunk_rows<D, 4>
                                          : k_chunk_rows<D, 8>;
        s = launch_dependent(rows, ctas, FR_WARPS * 32, 0, st, P);
    } else {
        ctas /= 2;
        s = launch_dependent(k_chunk_fma<D>, ctas, FC_NT, sizeof(FcSmem<D>), st, P);
    }
    if (s != HKV_OK)
        return s;
    return launch_dependent(k_chunk_merge<4, D>, merge_blocks(P, ctas), CMERGE_NT, 0, st, P);
}

}  // namespace hkv

using namespace hkv;

extern "C" {

hkv_status hkv_chunk_workspace_size(const hkv_problem *prob, int32_t tokens, size_t *bytes)
{
    const hkv_status s = check_problem(prob);
    if (s != HKV_OK)
        return s;
    if (tokens < 0 || tokens > HKV_MAX_TOKENS || bytes == nullptr)
        return HKV_ERR_INVALID_ARG;
    *bytes = chunk_ws(prob, tokens).total;
    return HKV_OK;
}

hkv_status hkv_chunk_attention(const hkv_problem *prob, const void *q, int64_t q_stride, int32_t tokens,
                               const int32_t *q_start, const int32_t *kv_len, const hkv_pages *pages, void *out,
                               float *lse, void *ws, size_t ws_bytes, hkv_stream_t stream)
{
    hkv_status s = check_problem(prob);
    if (s != HKV_OK)
        return s;
    if (prob->B > HKV_MAX_REQUESTS || tokens < 0 || tokens > HKV_MAX_TOKENS)
        return HKV_ERR_INVALID_ARG;
    if ((s = check_pages(pages, prob, true, true)) != HKV_OK)
        return s;
    const int es = es_of(prob->dtype), D = prob->D;
    const auto words = [](const void *p) { return p != nullptr && ptr_aligned(p, 4); };
    if (prob->B > 0 && (!words(q_start) || !words(kv_len)))
        return HKV_ERR_INVALID_ARG;
    if (tokens > 0 && (q == nullptr || out == nullptr || !ptr_aligned(q, 16) || !ptr_aligned(out, 16) ||
                       q_stride < (int64_t)prob->Hq * D || (q_stride * es) % 16))
        return HKV_ERR_INVALID_ARG;
    if (!ptr_aligned(lse, 4))
        return HKV_ERR_INVALID_ARG;
    if (tokens > 0) {
        const Span rows{q, ((tokens - 1) * q_stride + (int64_t)prob->Hq * D) * es};
        const Span o{out, (int64_t)tokens * prob->Hq * D * es}, l{lse, lse ? (int64_t)tokens * prob->Hq * 4 : 0};
        if (o.meets(rows) || l.meets(rows) || l.meets(o))
            return HKV_ERR_INVALID_ARG;
    }
    const ChunkWs w = chunk_ws(prob, tokens);
    if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < w.total)
        return HKV_ERR_WORKSPACE;
    if (tokens == 0 || prob->B == 0)
        return HKV_OK;
    ChunkP P{};
    P.q = static_cast<const char *>(q);
    P.qs = q_stride * es;
    P.q_start = q_start;
    P.kv_len = kv_len;
    P.pages = pages_p(pages, es);
    P.out = static_cast<char *>(out);
    P.lse = lse;
    char *base = static_cast<char *>(ws);
    P.part = reinterpret_cast<float *>(base + w.part);
    P.desc = reinterpret_cast<ChunkDesc *>(base + w.desc);
    P.B = prob->B;
    P.T = tokens;
    P.Hq = prob->Hq;
    P.Hkv = prob->Hkv;
    P.g_log2 = 31 - __builtin_clz((unsigned)(prob->Hq / prob->Hkv));
    P.rec_rows = w.rec_rows;
    P.scale_log2 = (prob->scale > 0.0f ? prob->scale : 1.0f / std::sqrt((float)D)) * 1.4426950408889634f;
    P.status = reinterpret_cast<uint32_t *>(base);
    P.wait_ns = g_wait_ns.load();
    P.withhold = g_withhold.load();
    const cudaStream_t st = (cudaStream_t)stream;
    if (prob->dtype == HKV_F32)
        return D == 128 ? run_fma<128>(P, w.ctas, st) : run_fma<64>(P, w.ctas, st);
    return D == 128 ? run_mma<128>(prob, P, w.ctas, st) : run_mma<64>(prob, P, w.ctas, st);
}

}  // extern "C"
