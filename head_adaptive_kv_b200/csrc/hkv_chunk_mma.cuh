// hkv_chunk_mma.cuh -- the chunk's attention in bf16 on the tensor cores.
//
// One CTA per SM, an item of 256 rows in two row tiles of 128, keys in tiles
// of 128. Scores S_t = Q_t K^T and outputs O_t += P_t V live in tensor memory
// (two of each fill its 512 columns at D = 128); the weights P_t overwrite S_t
// there as bf16 and are the product's A operand without touching shared
// memory. Warps:
//   0-3, 4-7  softmax of row tile 0, 1: a thread per row reads S, keeps the
//             row's maximum and sum, writes P; at the item's end reads O
//   8, 10     load Q, and K and V tiles page by page (tiled TMA) into a ring
//   9, 11     issue the matrix instructions of softmax group 0, 1
// The matrix instructions of one thread run in order, so S_t of the next key
// tile may be issued right behind the product that still reads P_t from the
// same columns, and a tile's softmax runs under the other tile's products. The
// two groups take turns at their exponentials: left alone they fall into step,
// share the exponential units and then leave them idle together (8192 tokens
// behind 8192, Hq 32, Hkv 8, D 128: 1.61 ms without turns, 1.43 with; taking
// part of the exponentials on the FMA units made it 1.45 to 1.53, at D = 64
// 1.15 to 1.17 instead of 1.13; scores in half tiles of 64 keys, two in flight,
// 1.53: narrow products cost as much as wide ones; at D = 64, P in columns of
// its own, so that scores need not wait for products, changed nothing). The
// weights go out in halves, so that the product with V begins before the last
// of them. At that size the card is at its power limit (1.64 GHz): 1.09 to 1.15
// of the 1.38 PFLOP/s that a library product sustains there. 64 single tokens
// on 4k to 32k keys: 6.8 TB/s in short runs, 6.0 at the power limit. The size of
// the pages does not matter much: 16 to 256 rows, the same within 1 %.
//
// Items of at most 128 rows (single tokens, short chunks) have one row tile;
// its key tiles then go to the two softmax groups in turn, each with its own
// O, joined at the item's end: two tiles in flight hide the softmax latency.
//
// The row maximum a weight refers to is only moved when a score passes it by
// 2^8, a known refinement of the running softmax (weights up to 2^8 are as
// exact as below 1, and fp32 sums hold them), so O is rarely rescaled.
//
// Every wait is bounded, a warp's lanes give up together, and what is under way
// then lands before the CTA ends.
#pragma once

#include <cuda_bf16.h>

#include "hkv_chunk.cuh"
#include "hkv_tcgen.cuh"

namespace hkv {

constexpr int CM_NT = 384;
constexpr int CM_M = 256, CM_NK = 128;
// (an item's start and end cost about two tiles: 2048 tokens alone 59 us, 62 counted as one, 59 as three)
using CmLine = ChunkLine<CM_M, CM_NK, 2, 2>;
constexpr float CM_GROW = 8.0f;  // log2 of the growth of a score that moves the reference

struct alignas(64) ChunkMmaP {
    ChunkP c;
    CUtensorMap q, q1, k, v;  // q1: boxes of one token's group
    int32_t none;  // a page coordinate outside the pool: the load gives zeros
};

template <int D>
struct CmSmem {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = 128 * D * 2;  // bytes of 128 rows
    static constexpr int NST = D == 128 ? 4 : 8;
    unsigned char q[2][TILE];
    unsigned char ring[NST][TILE];
    uint4 out[8][256];         // per softmax warp: 32 rows of 128 bytes on their way out
    uint64_t full[NST], empty[NST];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], o_full[2];
    uint64_t p_half[2], p_full[2];  // the weights of the tile's first 64 keys, of all
    uint64_t turn[2][4];            // a warp's exponentials may begin: the other group's warp beside it is through
    uint64_t x_ready, x_done;  // one row tile: group 1's statistics are there / its O has been read
    uint64_t drained[2];       // after a wait that ran out: the matrix instructions issued are done
    uint32_t items[2], issued[2];  // whose Q, and stages of the ring, a load warp has asked for
    uint32_t tmem;
    ChunkShare share;
    unsigned long long red[CM_NT / 32];
    float xm[128], xl[128];
};

// Position in a ring of N stages.
template <int N>
struct RingAt {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

// The item's last V tile holds rows behind the request's last token that take
// part in the product (it runs over whole groups of 16 keys, of the last item
// or of one that ends shortly before it): their weights are 0, but what lies
// there may be NaN. Rows from the item's limit on are zeroed.
__device__ __forceinline__ bool cm_tail(const ChunkWalk<CmLine> &it)
{
    return it.j1 == it.all && ((it.limit + 15) & ~15) > it.r.kv;
}

// ---- loads (warps 8 and 10) ---------------------------------------------------------------
//
// A tile's boxes (a page's rows by 64 columns) are issued by two warps in
// turn: a small box costs its issuer about as much as a large one.

template <int D>
__device__ __forceinline__ bool cm_load(const ChunkMmaP &P, CmSmem<D> &sm, const uint32_t limit, int lane, const int w)
{
    using SM = CmSmem<D>;
    const ChunkP &A = P.c;
    const PagesP &G = A.pages;
    const int rows = min(1 << G.page_log2, CM_NK);         // of a box
    const int per = CM_NK / rows;                          // boxes of a tile
    const uint32_t box = (uint32_t)rows * 128;             // bytes of a box
    RingAt<SM::NST> at;
    uint32_t items = 0, issued = 0;
    bool ok = true, bad = false;
    if (lane == 0)
        sm.items[w] = sm.issued[w] = 0;
    if (A.withhold)
        return true;
    for (ChunkWalk<CmLine> it(A, sm.share); it.item(); it.next()) {
        const int n = it.j1 - it.j0;
        if (n <= 0)
            continue;
        const int ahead = it.rows <= 128 ? 2 : 1;  // key tiles whose scores are formed ahead of a tile's product
        // this lane's table entry of tile j (lanes below `per`), looked at only when the tile is issued
        const auto page = [&](int j) {
            const int key = (it.j0 + j) * CM_NK + lane * rows;
            if (lane >= per || j >= n || key >= it.limit)
                return -1;
            return __ldg(G.table + it.b * G.table_stride + (key >> G.page_log2));
        };
        int next_k = page(0);
        ok = mbar_await(&sm.q_empty, (items & 1) ^ 1, limit);
        if (!ok)
            break;
        if (elect_one()) {
            const int tiles = it.rows <= 128 ? 1 : 2, toks = 128 >> A.g_log2;
            const bool single = it.rows == 1 << A.g_log2, mine = D == 128 || w == 0;
            mbar_arrive_expect_tx(&sm.q_full, !mine ? 0 : single ? it.rows * 128 : tiles * (128 * 128));
            if (mine) {
                // (a single token leaves the other rows as they were, zero as a rule: products of zeros cost no power)
                if (single)
                    tma_load3(sm.q[0] + w * (128 * 128), &P.q1, 64 * w, it.h << A.g_log2, it.row0, &sm.q_full);
                else
                    for (int t = 0; t < tiles; ++t)
                        tma_load3(sm.q[t] + w * (128 * 128), &P.q, 64 * w, it.h << A.g_log2, it.row0 + t * toks,
                                  &sm.q_full);
            }
        }
        __syncwarp();
        ++items;
        // the ring's order: K0 V0 K1 V1 ..., or with one row tile K0 K1 V0 K2 V1 ...
        int kj = 0, page0 = -1, page1 = -1;  // the pages of tiles vj and vj + 1
        for (int vj = 0; vj < n && ok;) {
            const bool is_k = kj < min(n, vj + ahead);
            const int j = is_k ? kj : vj, entry = is_k ? next_k : page0;
            if (is_k) {
                (kj == vj ? page0 : page1) = next_k;
                next_k = page(++kj);
            } else {
                page0 = page1;
                ++vj;
            }
            ok = mbar_await(&sm.empty[at.i], at.phase ^ 1, limit);
            if (!ok)
                break;
            uint64_t *bar = &sm.full[at.i];
            const int boxes = min(per, (it.limit - (it.j0 + j) * CM_NK + rows - 1) / rows);
            const bool lead = elect_one(), there = entry >= 0 && entry < G.pages;
            bad = bad || (w == 0 && lane < boxes && !there);
            // box i of columns 64 h is this warp's when i HALVES + h is of its parity
            if (lead)
                mbar_arrive_expect_tx(bar, (D == 128 ? boxes : (boxes + 1 - w) / 2) * box);
            const int row = (it.j0 + j) * CM_NK & ((1 << G.page_log2) - 1);  // a tile begins a page, or its second half
            unsigned char *dst = sm.ring[at.i] + (D == 128 ? w * (CM_NK * 128) : 0);
            const CUtensorMap *map = is_k ? &P.k : &P.v;
            // (one lane issues all its boxes: lanes that issue one each are served one after another, and slower)
            for (int i = D == 128 ? 0 : w; i < boxes; i += D == 128 ? 1 : 2) {
                const int pg = __shfl_sync(0xffffffffu, there ? entry : P.none, i);
                if (lead)
                    tma_load4(dst + i * rows * 128, map, D == 128 ? 64 * w : 0, row, it.h, pg, bar);
            }
            __syncwarp();
            at.next();
            ++issued;
        }
        if (!ok)
            break;
    }
    if (bad)
        atomicOr(A.status, HKV_DEV_BAD_INDEX);
    if (lane == 0) {
        sm.items[w] = items;
        sm.issued[w] = issued;
    }
    return ok;
}

// ---- matrix instructions (warps 9 and 11, one per softmax group) --------------------------
//
// The warp stays converged and one elected lane issues, so that descriptors
// live in uniform registers: a single warp issuing for both groups, or code in
// which one lane runs alone, could not keep the tensor cores fed.

template <int D>
__device__ __forceinline__ bool cm_issue(const ChunkMmaP &P, CmSmem<D> &sm, const uint32_t limit, const int g)
{
    using SM = CmSmem<D>;
    constexpr uint32_t ID_S = mma_idesc(CM_NK, false), ID_O = mma_idesc(D, true);
    const uint32_t ts = sm.tmem + g * 128, to = sm.tmem + 256 + g * 128;
    const uint32_t ring = mma_low(smem_addr(sm.ring[0]), 0), q0 = mma_low(smem_addr(sm.q[0]), 16);
    RingAt<SM::NST> at;
    uint32_t items = 0, p_count = 0;
    const auto landed = [&]() { return mbar_await(&sm.full[at.i], at.phase, limit); };
    // Both warps go past every stage and both free it (a parity wait that
    // skips phases, or one that a faster warp leaves two phases behind, would
    // be answered for the wrong one).
    const auto pass = [&]() {
        if (!landed())
            return false;
        if (elect_one())
            mbar_arrive(&sm.empty[at.i]);
        __syncwarp();
        at.next();
        return true;
    };
    // S = Q K^T with the present stage's K, which is then free
    const auto scores = [&](uint32_t q) {
        const uint32_t k = ring + at.i * (SM::TILE >> 4) + (1u << 16);
        if (elect_one()) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t off = (s / 4) * (128 * 128 >> 4) + (s % 4) * 2;
                mma_ss(ts, q + off, k + off, ID_S, s > 0);
            }
            mma_commit(&sm.s_full[g]);
            mma_commit(&sm.empty[at.i]);
        }
        __syncwarp();
        at.next();
    };
    // O (+)= P V with the stage's V, `keys` of whose keys (or all) count, in groups of 16, the first four as soon as
    // their weights are there; the stage is then free
    const auto product = [&](int stage, int keys, bool first, bool last, bool tail) {
        const int steps = (min(CM_NK, keys) + 15) / 16;
        if (tail) {
            // (both warps write the same zeros: neither waits for the other)
            const int gap = steps * 16 - keys;
            for (int i = threadIdx.x & 31; i < gap * 8 * SM::HALVES; i += 32) {
                const int half = i / (gap * 8), rest = i - half * gap * 8;
                *reinterpret_cast<uint4 *>(sm.ring[stage] + half * (CM_NK * 128) + (keys + rest / 8) * 128 +
                                           (rest % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
        const uint32_t v = ring + stage * (SM::TILE >> 4) + ((CM_NK * 128 >> 4) << 16);
        const auto some = [&](int from, int to_step) {
            for (int s = from; s < to_step; ++s)
                mma_ts(to, ts + s * 8, v + s * (2048 >> 4), ID_O, !(first && s == 0));
        };
        if (!mbar_await(&sm.p_half[g], p_count & 1, limit))
            return false;
        tc_fence_after();
        if (elect_one()) {
            if (steps >= 4) {
                mma_ts(to, ts, v, ID_O, !first);
#pragma unroll
                for (int s = 1; s < 4; ++s)
                    mma_ts(to, ts + s * 8, v + s * (2048 >> 4), ID_O, true);
            } else {
                some(0, steps);
            }
        }
        __syncwarp();
        if (!mbar_await(&sm.p_full[g], p_count & 1, limit))
            return false;
        ++p_count;
        tc_fence_after();
        if (elect_one()) {
            if (steps == 8) {
#pragma unroll
                for (int s = 4; s < 8; ++s)
                    mma_ts(to, ts + s * 8, v + s * (2048 >> 4), ID_O, true);
            } else {
                some(4, steps);
            }
            if (last)
                mma_commit(&sm.o_full[g]);
            mma_commit(&sm.empty[stage]);
        }
        __syncwarp();
        return true;
    };
    // this group's last scores of the item have been issued: Q is free when they are done
    const auto q_free = [&]() {
        if (elect_one())
            mma_commit(&sm.q_empty);
        __syncwarp();
    };
    for (ChunkWalk<CmLine> it(P.c, sm.share); it.item(); it.next()) {
        const int n = it.j1 - it.j0;
        if (n <= 0)
            continue;
        const bool one = it.rows <= 128;
        const auto keys = [&](int j) { return it.limit - (it.j0 + j) * CM_NK; };  // from tile j on
        const bool tail = cm_tail(it);
        if (!mbar_await(&sm.q_full, items & 1, limit))
            return false;
        ++items;
        if (one) {
            // ring: K0 K1 V0 K2 V1 ...; this group has the key tiles of its parity
            for (int j = 0; j < min(n, 2); ++j) {
                if (j != g) {
                    if (!pass())
                        return false;
                    continue;
                }
                if (!landed())
                    return false;
                tc_fence_after();
                scores(q0);
            }
            if (g + 2 >= n)
                q_free();
            for (int j = 0; j < n; ++j) {
                const bool mine = (j & 1) == g;
                if (!mine) {
                    if (!pass() || (j + 2 < n && !pass()))
                        return false;
                    continue;
                }
                if (!landed() || !product(at.i, keys(j), j < 2, j + 2 >= n, tail && j + 1 == n))
                    return false;
                at.next();
                if (j + 2 < n) {
                    if (!landed())
                        return false;
                    scores(q0);
                    if (j + 4 >= n)
                        q_free();
                }
            }
            continue;
        }
        // ring: K0 V0 K1 V1 ...; both groups use every tile
        const uint32_t q = q0 + g * (SM::TILE >> 4);
        if (!landed())
            return false;
        tc_fence_after();
        scores(q);
        if (n == 1)
            q_free();
        for (int j = 0; j < n; ++j) {
            const int vs = at.i;
            if (!landed())
                return false;
            at.next();
            if (j + 1 < n && !landed())
                return false;
            if (!product(vs, keys(j), j == 0, j + 1 == n, tail && j + 1 == n))
                return false;
            if (j + 1 < n) {
                scores(q);
                if (j + 2 == n)
                    q_free();
            }
        }
    }
    return true;
}

// ---- softmax and output (warps 0-7) -----------------------------------------------------

template <int D>
__device__ __forceinline__ bool cm_softmax(const ChunkMmaP &P, CmSmem<D> &sm, const uint32_t limit)
{
    const ChunkP &A = P.c;
    const int tid = threadIdx.x, group = tid / 128, row = tid % 128, lane = tid & 31, warp = row / 32;
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;  // this warp's quarter of the tensor memory
    const uint32_t ts = sm.tmem + group * 128 + lanes, to = sm.tmem + 256 + group * 128 + lanes;
    const float sc = A.scale_log2;
    const int G = 1 << A.g_log2;
    const int64_t rec = (int64_t)A.rec_rows * (D + 2);
    uint32_t s_count = 0, o_count = 0, x_count = 0, o_other = 0, turns = 0;  // phases; o_other: of group 1, seen from 0
    for (ChunkWalk<CmLine> it(A, sm.share); it.item(); it.next()) {
        if (!it.mine())
            continue;
        const int n = it.j1 - it.j0;
        const bool one = it.rows <= 128;
        const int r = one ? row : group * 128 + row;              // row of the item
        const bool warp_on = (r & ~31) < it.rows;                 // the warp has rows that are there
        const int seen = min(it.r.kv, it.pos0 + (r >> A.g_log2) + 1);  // keys the row sees
        const int least = min(it.r.kv, it.pos0 + ((r & ~31) >> A.g_log2) + 1);  // ... and the warp's first row
        float m = -INFINITY, l = 0.0f;
        bool begun = false;
        for (int j = one ? group : 0; j < n; j += one ? 2 : 1) {
            const int key0 = (it.j0 + j) * CM_NK;
            // pages of the tile that are not there (a bit per 16 keys)
            uint32_t holes = 0;
            if (warp_on) {
                const int key = key0 + (lane & 7) * 16;
                holes = __ballot_sync(0xffffffffu, key < it.limit && page_of(A.pages, it.b, key) < 0) & 0xffu;
            }
            if (!mbar_await(&sm.s_full[group], s_count & 1, limit))
                return false;
            ++s_count;
            if (warp_on) {
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmem_ld32(ts + 32 * i, s[i]);
                tmem_wait_ld();
                if (least - key0 < CM_NK || holes) {
                    const int cut = seen - key0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n_keep = max(0, min(32, cut - 32 * i));
                        uint32_t keep = n_keep == 32 ? 0xffffffffu : (1u << n_keep) - 1u;
                        keep &= ~(((holes >> (2 * i)) & 1u) * 0xffffu | ((holes >> (2 * i + 1)) & 1u) * 0xffff0000u);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((keep >> e) & 1u))
                                s[i][e] = 0xff800000u;  // -inf
                    }
                }
                float part[4];  // four chains: one would wait for itself 64 times
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    part[i] = __uint_as_float(s[i][0]);
#pragma unroll
                    for (int e = 1; e < 31; e += 2)
                        part[i] = fmaxf(part[i], fmaxf(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])));
                    part[i] = fmaxf(part[i], __uint_as_float(s[i][31]));
                }
                const float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                const bool grow = (top - m) * sc > CM_GROW;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2((m - top) * sc) : 1.0f;
                    if (grow)
                        m = top;
                    l *= f;
                    if (begun) {
                        // S of this tile was issued behind the product of the last: O is settled
#pragma unroll 1
                        for (int x = 0; x < D; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + x, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(to + x, o);
                        }
                    }
                }
                // (rows that are not there weigh nothing: zeros again)
                const float ref = r >= it.rows ? INFINITY : m == -INFINITY ? 0.0f : m * sc;
                const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
                float2 sum[2] = {make_float2(l, 0.0f), make_float2(0.0f, 0.0f)};
                // weights of columns 32 i .. 32 i + 31 as bf16 pairs
                const auto weigh = [&](int i, uint32_t *w) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = ffma2(make_float2(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])), sc2, ref2);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[(e / 2) & 1] = fadd2(sum[(e / 2) & 1], x);
                        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
                        w[e / 2] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                };
                if (!one && !mbar_await(&sm.turn[group][warp], (turns & 1) ^ (group == 0), limit))
                    return false;
                uint32_t w[32];
                weigh(0, w);
                weigh(1, w + 16);
                tmem_st32(ts, w);
                weigh(2, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.p_half[group]);
                weigh(3, w + 16);
                if (!one && lane == 0)
                    mbar_arrive(&sm.turn[group ^ 1][warp]);
                tmem_st32(ts + 32, w);
                const float2 both = fadd2(sum[0], sum[1]);
                l = both.x + both.y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
            } else {
                if (!one && !mbar_await(&sm.turn[group][warp], (turns & 1) ^ (group == 0), limit))
                    return false;
                if (lane == 0) {
                    mbar_arrive(&sm.p_half[group]);
                    if (!one)
                        mbar_arrive(&sm.turn[group ^ 1][warp]);
                }
            }
            turns += !one;
            begun = true;
            if (lane == 0)
                mbar_arrive(&sm.p_full[group]);
        }
        // the item's output (group 1 of a single row tile hands its part to group 0)
        const bool mine = begun;
        if (mine) {
            if (!mbar_await(&sm.o_full[group], o_count & 1, limit))
                return false;
            ++o_count;
        }
        if (!one && n > 0)
            ++o_other;
        const bool two_parts = one && n > 1;
        if (two_parts && group == 1) {
            sm.xm[row] = m;
            sm.xl[row] = l;
            mbar_arrive(&sm.x_ready);
            if (!mbar_await(&sm.x_done, x_count & 1, limit))
                return false;
            ++x_count;
            continue;
        }
        if (one && group == 1)
            continue;
        float fa = 1.0f, fb = 0.0f;
        if (two_parts) {
            if (!mbar_await(&sm.x_ready, x_count & 1, limit) || !mbar_await(&sm.o_full[1], o_other & 1, limit))
                return false;
            ++x_count;
            ++o_other;
            const float m1 = sm.xm[row], l1 = sm.xl[row], M = fmaxf(m, m1), base = M == -INFINITY ? 0.0f : M;
            fa = ex2((m - base) * sc);
            fb = ex2((m1 - base) * sc);
            l = l * fa + l1 * fb;
            m = M;
        }
        const bool whole = it.whole();
        const bool valid = r < it.rows;
        const auto row_at = [&](int x) {  // row x of the item in out and lse
            return ((int64_t)it.row0 + (x >> A.g_log2)) * A.Hq + (it.h << A.g_log2) + (x & (G - 1));
        };
        float *record = A.part + (2 * (int64_t)blockIdx.x + (it.first_part() ? 1 : 0)) * rec;
        if (warp_on) {
            tc_fence_after();
            if (whole) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                fa *= inv;
                fb *= inv;
            }
            const bool any = l > 0.0f;
            // 32 output columns of this row
            const auto columns = [&](int x, uint32_t (&o)[32]) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = 0u;
                if (mine) {
                    tmem_ld32(to + x, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * fa) : 0u;
                }
                if (two_parts) {
                    uint32_t o1[32];
                    tmem_ld32(to + 128 + x, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (any)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), fb, __uint_as_float(o[e])));
                }
            };
            // Each thread has a row; memory wants rows from neighbouring lanes. Eight pieces of 16 bytes a row
            // pass through shared memory, piece p of row y at p ^ (y mod 8): no two lanes of a quarter warp meet
            // in a bank, on the way in or out.
            uint4 *stage = sm.out[tid / 32];
            const int first = r & ~31;  // the warp's first row of the item
            const auto pass_on = [&](char *base, int64_t stride, bool to_record) {
                __syncwarp();
                const int rows = min(32, it.rows - first);
#pragma unroll 1
                for (int y = lane / 8; y < rows; y += 16) {
                    const int p = lane % 8;
                    // four rows at once: the loads of shared memory are on their way together
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        if (y + i < rows)
                            *reinterpret_cast<uint4 *>(
                                base + (to_record ? first + y + i : row_at(first + y + i)) * stride + p * 16) =
                                stage[8 * (y + i) + (p ^ ((y + i) & 7))];
                }
                __syncwarp();
            };
            // (loops, not copies: code that runs once an item comes from far away each time)
            if (whole) {
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    columns(x, o);
                    const int half = x & 32 ? 4 : 0;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * i]),
                                                                           __uint_as_float(o[e + 2 * i + 1]));
                            w[i] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        stage[8 * lane + ((half + e / 8) ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (half)
                        pass_on(A.out + (x - 32) * 2, D * 2, false);
                }
            } else {
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    columns(x, o);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        stage[8 * lane + ((e / 4) ^ (lane & 7))] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    pass_on(reinterpret_cast<char *>(record + x), D * 4, true);
                }
            }
            tc_fence_before();
            if (valid) {
                if (!whole) {
                    record[(int64_t)A.rec_rows * D + r] = m == -INFINITY ? m : m * sc;
                    record[(int64_t)A.rec_rows * (D + 1) + r] = l;
                } else if (A.lse != nullptr) {
                    A.lse[row_at(r)] = l > 0.0f ? (m * sc + log2f(l)) * 0.6931471805599453f : -INFINITY;
                }
            }
        }
        if (two_parts)
            mbar_arrive(&sm.x_done);
        if (tid == 0 && !whole && it.first_part())
            A.desc[blockIdx.x] = ChunkDesc{it.parts(), it.row0, it.h, it.rows};
    }
    return true;
}

template <int D>
__global__ void __launch_bounds__(CM_NT, 1) k_chunk_mma(const __grid_constant__ ChunkMmaP P)
{
    extern __shared__ unsigned char smem_raw[];
    auto &sm = *reinterpret_cast<CmSmem<D> *>(smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_dependents();  // only the merge follows, which waits for this kernel's end
    if (tid == 0) {
        for (int i = 0; i < CmSmem<D>::NST; ++i) {
            mbar_init(&sm.full[i], 2);
            mbar_init(&sm.empty[i], 2);
        }
        mbar_init(&sm.q_full, 2);
        mbar_init(&sm.q_empty, 2);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&sm.s_full[g], 1);
            mbar_init(&sm.p_half[g], 4);
            mbar_init(&sm.p_full[g], 4);
            for (int w = 0; w < 4; ++w)
                mbar_init(&sm.turn[g][w], 1);
            mbar_init(&sm.o_full[g], 1);
        }
        mbar_init(&sm.x_ready, 128);
        mbar_init(&sm.x_done, 128);
        mbar_init(&sm.drained[0], 1);
        mbar_init(&sm.drained[1], 1);
        mbar_fence_init();
    }
    if (warp == 9)
        tmem_alloc(&sm.tmem, 512);
    if (warp == 8 && lane < 4)
        tma_prefetch_map(lane == 0 ? &P.q : lane == 1 ? &P.k : lane == 2 ? &P.v : &P.q1);
    for (int i = tid; i < (int)sizeof(sm.q[0]) / 16; i += CM_NT)
        reinterpret_cast<uint4 *>(sm.q[0])[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    wait_prior_grid();
    const uint32_t limit = await_limit(P.c.wait_ns);
    if (tid == 0)
        P.c.desc[blockIdx.x].n = 0;
    tc_fence_before();
    chunk_share<CM_NT, CmLine>(P.c, sm.red, &sm.share);  // (its barriers publish the set-up above)
    __syncthreads();
    tc_fence_after();
    // the launch's 384 x 168 registers, as 256 x 208 + 128 x 88: a softmax thread holds a row of S
    bool through;  // no wait of this warp has run out
    if (warp < 8) {
        regs_take<208>();
        through = cm_softmax<D>(P, sm, limit);
    } else {
        regs_give<88>();
        if (warp == 8 || warp == 10)
            through = cm_load<D>(P, sm, limit, lane, warp == 10);
        else
            through = cm_issue<D>(P, sm, limit, warp == 11);
    }
    tc_fence_before();
    if (!__syncthreads_and(through)) {
        // Somebody's wait has run out, so not all that is under way has been waited for, not even by warps that came
        // through: loads, products and weights land before the CTA ends.
        if (tid == 0)
            atomicOr(P.c.status, HKV_DEV_TIMEOUT);
        if (warp < 8) {
            tmem_wait_st();
        } else if (warp == 8 || warp == 10) {
            constexpr uint32_t NST = CmSmem<D>::NST;
            const uint32_t items = sm.items[warp == 10], issued = sm.issued[warp == 10];
            for (uint32_t i = issued < NST ? 0 : issued - NST; i < issued; ++i)
                mbar_let_land(&sm.full[i % NST], (i / NST) & 1);
            if (items > 0)
                mbar_let_land(&sm.q_full, (items - 1) & 1);
        } else {
            if (elect_one())
                mma_commit(&sm.drained[warp == 11]);
            mbar_let_land(&sm.drained[warp == 11], 0);
        }
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 9) {
        tc_fence_after();
        tmem_free(sm.tmem, 512);
    }
}

}  // namespace hkv
