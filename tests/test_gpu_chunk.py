"""GPU parity of the chunk's attention over the paged cache against the 64-bit oracle, and the whole prompt side run
together with the decode step."""
import numpy as np
import pytest
import torch

import oracle
from head_adaptive_kv_b200 import hkv, prompt
from head_adaptive_kv_b200.workloads import to_host_bits
from oracle import prompt as op
from tests import gpu_helpers as H
from tests.prompt_helpers import attention_bounds, f64, norm_bounds, pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


class Case:
    def __init__(self, lens, Hq, Hkv, D, dtype, page, layout="hnd", pad=0, seed=0, std=1.0, scale=0.0, cols=None):
        """lens: (cached, new) of each request; pad: rows behind the last."""
        rng = np.random.default_rng(seed)
        self.kv = [c + n for c, n in lens]
        self.starts = np.cumsum([0] + [n for _, n in lens])
        B, T = len(lens), int(self.starts[-1]) + pad
        self.k, self.v, self.table = pool(rng, B, self.kv, Hkv, D, page, dtype, layout=layout, device=DEV, cols=cols)
        g = torch.Generator().manual_seed(seed + 1)
        wide = (torch.randn(T, Hq * D + 24, generator=g) * 2 * std).to(dtype).to(DEV)
        self.q = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
        self.prob = hkv.Problem(B, Hq, Hkv, D, dtype, 1.0, 0, 0, scale=scale)
        self.page, self.bf16, self.T = page, dtype == BF, T
        self.scale = scale or D ** -0.5
        self.ws = prompt.ChunkWorkspace(self.prob, T, DEV)
        self.q_start, self.kv_len = i32(self.starts), i32(self.kv)
        self.out = torch.full((T, Hq, D), 5.0, dtype=dtype, device=DEV)
        self.lse = torch.full((T, Hq), 5.0, device=DEV)

    def run(self, lse=True, ws=None, out=None):
        prompt.chunk_attention(self.prob, self.q, self.q_start, self.kv_len, prompt.Pages(self.k, self.v, self.table),
                               self.out if out is None else out, ws or self.ws, lse=self.lse if lse else None)
        return self

    def reference(self):
        clean = lambda x: np.nan_to_num(f64(x), nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
        return op.chunk_attention(clean(self.q), clean(self.k), clean(self.v), self.q_start.cpu().numpy(),
                                  self.kv_len.cpu().numpy(), self.table.cpu().numpy(), self.page, self.scale)

    def check(self, status=0):
        assert self.ws.status() == status
        n = int(self.q_start[-1])
        ref = self.reference()
        tol, lse_tol = attention_bounds(ref, self.bf16)
        err = np.abs(f64(self.out) - ref[0])[:n]
        assert np.isfinite(err).all() and (err <= tol[:n]).all(), (err.max(), (err / tol[:n]).max())
        got, want = f64(self.lse)[:n], ref[1][:n]
        none = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), none)
        assert (np.abs(got[~none] - want[~none]) <= lse_tol[:n][~none]).all()
        assert (self.out[n:] == 5.0).all() and (self.lse[n:] == 5.0).all()  # rows behind the last sequence


MIXED = [(0, 1), (5, 1), (300, 1), (0, 70), (17, 64), (129, 33), (0, 0), (40, 0), (1000, 3), (127, 1), (128, 129)]
SHAPES = [(BF, 8, 2, 128, 16), (BF, 4, 4, 64, 32), (BF, 8, 1, 128, 64), (BF, 4, 2, 64, 128), (BF, 2, 2, 128, 256),
          (BF, 16, 2, 64, 16), (F32, 4, 2, 64, 16), (F32, 8, 2, 128, 64), (F32, 2, 2, 128, 256), (F32, 8, 1, 64, 32)]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page", SHAPES)
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_mixed_batch(dtype, Hq, Hkv, D, page, layout):
    Case(MIXED, Hq, Hkv, D, dtype, page, layout, pad=5, seed=page).run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [
    [(0, 1)], [(1, 1)], [(127, 1)], [(128, 1)], [(4999, 1)],             # single tokens, the cache split over CTAs
    [(0, 2)], [(0, 63)], [(0, 64)], [(0, 65)], [(0, 128)], [(0, 129)],   # whole prompts around the tile edges
    [(0, 257)], [(63, 257)], [(1111, 37)], [(3000, 200)],
    [(777, 1)] * 9, [(i * 13, 1) for i in range(60)],                    # decode batches
], ids=lambda x: f"{len(x)}x{x[0]}")
def test_lengths(dtype, lens):
    Case(lens, 8, 2, 128, dtype, 64, seed=len(lens)).run().check()


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_groups(G, D):
    for dtype in (BF, F32):
        Case([(200, 100), (0, 300), (700, 2)], 2 * G, 2, D, dtype, 32, seed=G).run().check()


def test_large_and_small_logits():
    # scores far apart (one key takes all) and all alike; an explicit scale
    for dtype in (BF, F32):
        Case([(300, 70)], 4, 2, 128, dtype, 32, std=6.0, seed=1).run().check()
        Case([(300, 70)], 4, 2, 128, dtype, 32, std=0.0, seed=2).run().check()
        Case([(300, 70)], 4, 2, 64, dtype, 16, scale=0.31, seed=3).run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_growing_scores(dtype):
    """Keys whose scores rise along the cache: the running maximum moves at every tile."""
    c = Case([(1500, 40)], 4, 2, 128, dtype, 64, seed=4)
    ids = c.table[0].long()
    step = torch.arange(ids.numel() * 64, device=DEV) / 200.0
    q = c.q.float().mean((0, 1))
    dirn = (q / q.norm()).to(dtype)
    c.k[ids] = c.k[ids] * 0.2 + (step.view(-1, 1, 64, 1) * dirn * 4).to(dtype)
    c.q.copy_(c.q * 0.2 + dirn * 8)
    c.run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 128])
def test_what_lies_behind_the_lengths_may_be_anything(dtype, page):
    c = Case([(50, 1), (120, 9), (0, 3), (255, 1), (128, 1)], 8, 2, 128, dtype, page, pad=40, seed=6)
    for b, L in enumerate(c.kv):
        for j in range(L, -(-L // page) * page):
            p = int(c.table[b, j // page])
            c.k[p, :, j % page] = float("nan") if j % 2 else float("inf")
            c.v[p, :, j % page] = float("inf") if j % 2 else float("nan")
    used = set(c.table[c.table >= 0].tolist())
    for p in range(c.k.shape[0]):
        if p not in used:
            c.k[p], c.v[p] = float("nan"), float("nan")
    c.q[int(c.starts[-1]):] = float("nan")
    c.run().check()


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_last_tokens_of_a_chunk_alone_in_an_item(dtype, G):
    """The last item of the chunk is 1 to 15 tokens, and the one before ends within 16 keys of what lies behind."""
    tokens = (256 if dtype == BF else 64) // G  # of an item
    c = Case([(42 + i, tokens + i) for i in (1, 3, 9, 15)] + [(0, 2 * tokens + 5)], 2 * G, 2, 64, dtype, 128, seed=24)
    for b, L in enumerate(c.kv):
        if L % 128:
            p = int(c.table[b, L // 128])
            c.k[p, :, L % 128:], c.v[p, :, L % 128:] = float("nan"), float("nan")
    c.run().check()


def test_one_request_full_of_nan_spoils_no_other():
    lens = [(100, 5), (60, 7), (30, 1)]
    for dtype in (BF, F32):
        c = Case(lens, 8, 2, 64, dtype, 16, seed=7).run()
        want = c.out.clone()
        ids = c.table[1, :5].long()
        c.k[ids], c.v[ids] = float("nan"), float("nan")
        c.q[5:12] = float("nan")
        c.run()
        torch.cuda.synchronize()
        keep = [0, 1, 2, 3, 4, 12]
        assert torch.equal(c.out[keep], want[keep])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_that_are_not_there(dtype):
    c = Case([(100, 40), (20, 30), (0, 20), (300, 1)], 4, 2, 128, dtype, 16, seed=8)
    n = c.k.shape[0]
    for b, col, bad in ((0, 2, -1), (0, 8, n), (1, 0, 2**31 - 1), (1, 1, -5), (2, 0, -1), (2, 1, -1), (3, 7, n + 3)):
        c.table[b, col] = bad
    c.run().check(hkv.DEV_BAD_INDEX)
    assert (c.out[70:86] == 0).all() and torch.isneginf(c.lse[70:86]).all()  # rows that see nothing


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_without_keys_and_lengths_out_of_range(dtype):
    # fewer cached tokens than new rows: the first rows see nothing (no clamp: the call can be made)
    c = Case([(0, 30), (50, 20)], 4, 2, 64, dtype, 16, seed=9)
    c.kv_len.copy_(i32([7, 0]))
    c.kv = [7, 0]
    c.run().check()
    assert (c.out[:23] == 0).all() and torch.isneginf(c.lse[30:]).all()
    # beyond the table's columns, below zero, and rows beyond the buffer
    c = Case([(0, 30), (50, 20)], 4, 2, 64, dtype, 16, seed=9)
    c.kv_len.copy_(i32([10**9, -3]))
    c.q_start.copy_(i32([-5, 30, 10**6]))
    c.table[:, 2:] = c.table[1, 2:].clone()
    c.run()
    assert c.ws.status() == hkv.DEV_LEN_CLAMPED
    c.kv_len.copy_(i32([c.table.shape[1] * 16, 0]))
    c.q_start.copy_(i32([0, 30, 50]))
    c.check()
    # descending starts
    c.q_start.copy_(i32([20, 10, 10]))
    c.run()
    assert c.ws.status() == hkv.DEV_LEN_CLAMPED


def test_nothing_to_do():
    c = Case([(10, 0), (0, 0)], 4, 2, 64, BF, 16, pad=3).run()
    c.check()
    c = Case([(10, 0)], 4, 2, 64, F32, 16).run()
    assert c.ws.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_every_time_and_without_lse(dtype):
    c = Case([(900, 1), (10, 300), (2000, 5)], 8, 2, 128, dtype, 32, seed=10).run()
    a = c.out.clone()
    for _ in range(3):
        c.out.zero_()
        c.run(lse=False)
        assert torch.equal(c.out, a)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_prompt_in_chunks_is_the_prompt(dtype):
    """One call over the prompt, and calls over its pieces: each piece within the bounds of the same oracle rows."""
    c = Case([(0, 333)], 8, 2, 128, dtype, 32, seed=11)
    ref = c.reference()
    tol, _ = attention_bounds(ref, c.bf16)
    for a, e in ((0, 1), (1, 2), (2, 130), (130, 131), (131, 333)):
        out = torch.zeros(e - a, 8, 128, dtype=dtype, device=DEV)
        prompt.chunk_attention(c.prob, c.q[a:e], i32([0, e - a]), i32([e]), prompt.Pages(c.k, c.v, c.table), out, c.ws)
        assert (np.abs(f64(out) - ref[0][a:e]) <= tol[a:e]).all()
    assert c.ws.status() == 0


def test_other_stream_and_two_calls_at_once():
    a, b = (Case([(700, 1), (3, 200)], 8, 2, 128, BF, 64, seed=s) for s in (12, 13))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replays_follow_the_lengths(dtype):
    """One captured call, replayed for other lengths of the same batch, and a second graph on the same workspace."""
    c = Case([(600, 30), (80, 64), (0, 50)], 8, 2, 128, dtype, 16, seed=14)
    c.run()
    torch.cuda.synchronize()
    other = torch.zeros_like(c.out)
    graphs = []
    for out in (c.out, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out)
        graphs.append(g)
    for kv, starts in (([630, 144, 50], [0, 30, 94, 144]), ([100, 144, 7], [0, 1, 94, 101]), ([1, 1, 1], [0, 1, 2, 3])):
        c.kv_len.copy_(i32(kv))
        c.q_start.copy_(i32(starts))
        c.out.fill_(5.0), c.lse.fill_(5.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        c.check()
        assert torch.equal(other[:starts[-1]], c.out[:starts[-1]])


def test_rows_far_into_the_pool():
    """Pages whose byte offsets pass 32 bits."""
    pages, Hkv, page, D = 70000, 4, 64, 128  # 4.6 GB each of K and V
    k, v = (torch.empty(pages, Hkv, page, D, dtype=BF, device=DEV) for _ in range(2))
    c = Case([(200, 5), (90, 1)], 8, Hkv, D, BF, page, seed=15)
    far = torch.arange(c.k.shape[0], device=DEV)
    far = torch.where(far % 2 == 0, pages - 1 - far, 33000 + far)
    k[far], v[far] = c.k, c.v
    small = c.table.clone()
    c.table.copy_(torch.where(small >= 0, far[small.clamp(min=0).long()].to(torch.int32), -1))
    near = c.k, c.v
    c.k, c.v = k, v
    c.run()
    c.k, c.v, c.table = near[0], near[1], small
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_to_decode(dtype):
    """The prompt side run together, as a serving loop does: two requests' prompts in chunks through plan, norms and
    rotation, attention; then the tiers are filled, the pages go back, and decode steps follow (norms, append, step).
    Attention over every token (p = 1, no clamp) makes the decode step's output that of plain attention."""
    Hq, Hkv, D, page, B = 8, 2, 64, 16, 2
    bf16 = dtype == BF
    lens, steps = [150, 83], 3
    pieces = [(64, 83), (50, 0), (36, 0)]  # tokens of each request in each step
    prob = hkv.Problem(B, Hq, Hkv, D, dtype, 1.0, 0, 512)
    g = torch.Generator().manual_seed(16)
    qkv = [(torch.randn(n + steps, (Hq + 2 * Hkv) * D, generator=g)).to(dtype).to(DEV) for n in lens]
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(dtype).to(DEV) for _ in range(2))
    rope = prompt.Rope.of_base(D, 1e4, DEV)
    T = 160
    state, ch = prompt.PageState.allocate(B, 12, page, 20, DEV), prompt.Chunk.allocate(B, T, DEV)
    pk, pv = (torch.full((20, Hkv, page, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    pages, ws = prompt.Pages(pk, pv, state.table), prompt.ChunkWorkspace(prob, T, DEV)
    heads = [Hq * D, Hkv * D, Hkv * D]
    q_all = [[] for _ in lens]
    outs = [[] for _ in lens]
    ctx, at = i32([0, 0]), [0, 0]
    for new in pieces:
        prompt.page_plan(ctx, i32(new), state, state, ch, ws)
        rows = torch.zeros(T, sum(heads), dtype=dtype, device=DEV)
        i = 0
        for b, n in enumerate(new):
            rows[i:i + n] = qkv[b][at[b]:at[b] + n]
            i += n
        q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split(heads, 1))
        qo, out = torch.zeros(T, Hq, D, dtype=dtype, device=DEV), torch.zeros(T, Hq, D, dtype=dtype, device=DEV)
        prompt.qk_norm_rope(prob, q, k, v, ch.pos, rope, qo, ws, q_weight=qw, k_weight=kw, pages=pages, slot=ch.slot)
        prompt.chunk_attention(prob, qo, ch.q_start, ch.kv_len, pages, out, ws)
        i = 0
        for b, n in enumerate(new):
            q_all[b].append(qo[i:i + n])
            outs[b].append(out[i:i + n])
            at[b] += n
            i += n
        ctx = ch.kv_len.clone()
    assert ws.status() == 0 and ctx.tolist() == lens
    # the cache holds what the oracle says, and each row's attention is the oracle's over it
    kc, vc, qs = [], [], []
    for b, n in enumerate(lens):
        ids = state.table[b].long()
        kb, vb = (x[ids.clamp(min=0)].transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for x in (pk, pv))
        x = qkv[b][:n].unflatten(1, (-1, D))
        pos, f = np.arange(n), f64(rope.inv_freq)
        ref, mag = op.norm_rope(f64(x[:, Hq:Hq + Hkv]), f64(kw), pos, f, D, False, 1.0, 1e-6)
        assert (np.abs(f64(kb.transpose(0, 1)) - ref) <= norm_bounds(ref, mag, bf16)).all()
        assert torch.equal(vb.transpose(0, 1), x[:, Hq + Hkv:])
        ref = op.chunk_attention(f64(torch.cat(q_all[b])), f64(pk.nan_to_num()), f64(pv.nan_to_num()), [0, n], [n],
                                 state.table[b:b + 1].cpu().numpy(), page, D ** -0.5)
        tol, _ = attention_bounds(ref, bf16)
        assert (np.abs(f64(torch.cat(outs[b])) - ref[0]) <= tol).all()
        kc.append(kb.clone()), vc.append(vb.clone())
    # hand over to the tiers
    tier = lambda n: hkv.Tier(torch.zeros(B, Hkv, n, D, dtype=dtype, device=DEV),  # noqa: E731
                              torch.zeros(B, Hkv, n, D, dtype=dtype, device=DEV), i32([0] * B * Hkv))
    dense, sparse, head = tier(32), tier(200), i32([0] * B * Hkv)
    prompt.fill_tiers(prob, pages, ch.kv_len, dense, head, sparse, ws)
    prompt.page_release(i32([1, 1]), state, state, ws)
    assert int(state.free_count) == 20 and state.held.tolist() == [0, 0]
    pk.fill_(float("nan")), pv.fill_(float("nan"))  # the pages belong to others now
    sws = hkv.Workspace(prob, dense, sparse, None)
    so = hkv.StepOutputs.allocate(prob, sparse, DEV)
    for step in range(steps):
        x = torch.stack([qkv[b][lens[b] + step] for b in range(B)])
        q, k, v = (y.unflatten(1, (-1, D)) for y in x.split(heads, 1))
        qo, kn, vn = torch.empty(B, Hq, D, dtype=dtype, device=DEV), *(torch.empty(B, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
        prompt.qk_norm_rope(prob, q, k, v, i32([n + step for n in lens]), rope, qo, ws, q_weight=qw, k_weight=kw, k_out=kn,
                            v_out=vn)
        hkv.append(prob, kn, vn, dense, head, sparse, sws)
        hkv.step(prob, qo, dense, sparse, None, so, sws)
        for b in range(B):
            kc[b], vc[b] = torch.cat([kc[b], kn[b][:, None]], 1), torch.cat([vc[b], vn[b][:, None]], 1)
            s = torch.einsum("hgd,hnd->hgn", qo[b].double().view(Hkv, -1, D), kc[b].double()) * D ** -0.5
            want = torch.einsum("hgn,hnd->hgd", s.softmax(-1), vc[b].double()).reshape(Hq, D)
            assert (so.out[b].double() - want).abs().max() <= H.ATOL
    assert ws.status() == 0 and sws.status() == 0


def test_waits_that_run_out_end_the_call():
    """Loads withheld: every wait of the kernel runs out, it returns, the status word says so, and after the workspace is
    zeroed again the next call is right."""
    c = Case([(300, 40), (20, 1)], 8, 2, 128, BF, 32, seed=17)
    hkv.set_wait_limit_ns(2_000_000)
    hkv.debug_withhold_publish(True)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        hkv.debug_withhold_publish(False)
        hkv.set_wait_limit_ns(1_000_000_000)
    assert c.ws.status() == hkv.DEV_TIMEOUT
    c.ws.init()
    c.out.fill_(5.0), c.lse.fill_(5.0)
    c.run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_requests(dtype):
    """More requests than a CTA has threads: single tokens, some requests without any, and a mixed batch."""
    single = [(7 * i % 300, 0 if i % 11 == 5 else 1) for i in range(900)]
    Case(single, 2, 2, 64, dtype, 16, seed=18).run().check()
    mixed = [(5 * i % 40, 1 + i % 3) for i in range(800)]
    Case(mixed, 2, 1, 64, dtype, 16, seed=19).run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_most_requests(dtype):
    """8192 requests, the limit of a call."""
    Case([(3 * i % 50, 0 if i % 7 == 3 else 1) for i in range(8192)], 2, 2, 64, dtype, 16, seed=31).run().check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(32767, 1)], [(16384, 32)], [(20000, 1), (12000, 45), (9, 1)]], ids=lambda x: f"{len(x)}x{x[0]}")
def test_items_in_more_parts_than_a_warp_has_lanes(lens, D):
    """One KV head: a few items on long contexts, each cut over a hundred CTAs or so and joined 32 records at a time."""
    for dtype in (BF, F32):
        Case(lens, 8, 1, D, dtype, 128, seed=32).run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_single_tokens_in_a_batch_of_more_rows(dtype):
    """Rows above the requests' count pick the kernel for chunks; the lengths may be single tokens all the same, and
    fewer rows than requests may hold one longer chunk."""
    c = Case([(500, 1), (0, 1), (90, 1)], 8, 2, 128, dtype, 32, pad=200, seed=20)
    c.run().check()
    Case([(500, 3), (40, 0), (90, 0), (7, 0)], 8, 2, 128, dtype, 32, seed=21).run().check()


def test_an_empty_pool():
    for dtype in (BF, F32):
        c = Case([(3, 2), (0, 1)], 4, 2, 64, dtype, 16, seed=22)
        c.k, c.v = c.k[:0], c.v[:0]
        c.run()
        assert c.ws.status() == hkv.DEV_BAD_INDEX
        assert (c.out == 0).all() and torch.isneginf(c.lse).all()


def test_one_row_of_any_stride():
    c = Case([(40, 1)], 8, 2, 128, BF, 32, seed=23)
    wide = torch.zeros(1, 8 * 128 + 3, dtype=BF, device=DEV)
    wide[:, :1024] = c.q.reshape(1, 1024)
    c.q = wide[:, :1024].unflatten(1, (8, 128))
    c.run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_requests_that_share_pages(dtype):
    """A prefix's pages stand in several tables, and one page twice in the same table."""
    c = Case([(96, 3), (96, 40), (64, 1), (200, 1)], 8, 2, 128, dtype, 32, seed=24)
    c.table[1, :3] = c.table[0, :3]
    c.table[2, :2] = c.table[0, :2]
    c.table[3, 1] = c.table[3, 0]
    c.run().check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_loop(dtype):
    """Plan, norms and attention as one graph, replayed for steps of other lengths while the state and the lengths
    advance in place, leaves the same bits as the calls one by one; the tiers of what finished come from a second
    graph on the same workspace, with the release."""
    Hq, Hkv, D, page, B, T, pool_pages = 8, 2, 128, 16, 4, 128, 40
    prob = hkv.Problem(B, Hq, Hkv, D, dtype, 1.0, 0, 0)
    gen = torch.Generator().manual_seed(25)
    steps = [([60, 0, 5, 0], [0, 0, 0, 0]), ([1, 40, 70, 0], [0, 0, 0, 0]), ([1, 1, 1, 1], [0, 1, 0, 1]),
             ([0, 0, 0, 0], [0, 0, 1, 0]), ([17, 9, 100, 2], [1, 0, 0, 0])]
    rows = [torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen).to(dtype).to(DEV) for _ in steps]
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(dtype).to(DEV)
    rope = prompt.Rope.of_base(D, 1e4, DEV)

    class Loop:
        def __init__(self):
            self.state = prompt.PageState.allocate(B, 16, page, pool_pages, DEV)
            self.ch = prompt.Chunk.allocate(B, T, DEV)
            pk, pv = (torch.zeros(pool_pages, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2))
            self.pages, self.ws = prompt.Pages(pk, pv, self.state.table), prompt.ChunkWorkspace(prob, T, DEV)
            self.x = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=dtype, device=DEV)
            self.new, self.done = i32([0] * B), i32([0] * B)
            self.q, self.out = (torch.zeros(T, Hq, D, dtype=dtype, device=DEV) for _ in range(2))
            tier = lambda n: hkv.Tier(torch.zeros(B, Hkv, n, D, dtype=dtype, device=DEV),  # noqa: E731
                                      torch.zeros(B, Hkv, n, D, dtype=dtype, device=DEV), i32([0] * B * Hkv))
            self.dense, self.sparse, self.head = tier(24), tier(160), i32([0] * B * Hkv)

        def step(self):
            prompt.page_plan(self.ch.kv_len, self.new, self.state, self.state, self.ch, self.ws)
            q, k, v = (y.unflatten(1, (-1, D)) for y in self.x.split([Hq * D, Hkv * D, Hkv * D], 1))
            prompt.qk_norm_rope(prob, q, k, v, self.ch.pos, rope, self.q, self.ws, q_weight=w, k_weight=w,
                                pages=self.pages, slot=self.ch.slot)
            prompt.chunk_attention(prob, self.q, self.ch.q_start, self.ch.kv_len, self.pages, self.out, self.ws)

        def finish(self):
            prompt.fill_tiers(prob, self.pages, self.ch.kv_len, self.dense, self.head, self.sparse, self.ws,
                              take=self.done)
            prompt.page_release(self.done, self.state, self.state, self.ws)
            self.ch.kv_len.mul_(1 - self.done)

        def results(self):
            return [self.state.table, self.state.free, self.state.free_count, self.state.held, self.ch.q_start,
                    self.ch.kv_len, self.ch.pos, self.ch.slot, self.q, self.out, self.pages.k, self.pages.v,
                    self.dense.k, self.dense.v, self.dense.len, self.sparse.k, self.sparse.v, self.sparse.len, self.head]

    eager, replayed = Loop(), Loop()
    for loop in (eager, replayed):  # no requests yet: nothing moves
        loop.step(), loop.finish()
    torch.cuda.synchronize()
    graphs = []
    for call in (replayed.step, replayed.finish):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for (new, done), x in zip(steps, rows):
        for loop in (eager, replayed):
            loop.new.copy_(i32(new)), loop.done.copy_(i32(done)), loop.x.copy_(x)
        eager.step(), eager.finish()
        graphs[0].replay(), graphs[1].replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.results(), replayed.results()):
            assert torch.equal(a, b)
    assert eager.ws.status() == 0 and replayed.ws.status() == 0
    held = [-(-n // page) for n in eager.ch.kv_len.tolist()]
    assert eager.state.held.tolist() == held and int(eager.state.free_count) == pool_pages - sum(held)
    assert sorted(eager.state.free[:pool_pages - sum(held)].tolist()
                  + [p for b, h in enumerate(held) for p in eager.state.table[b, :h].tolist()]) == list(range(pool_pages))


def test_the_whole_side_on_two_streams_at_once():
    """Two loops of plan, norms, attention and fill, each on a stream and a workspace of its own."""
    Hq, Hkv, D, page, B, T = 8, 2, 64, 32, 3, 300
    prob = hkv.Problem(B, Hq, Hkv, D, BF, 1.0, 0, 0)
    rope = prompt.Rope.of_base(D, 1e4, DEV)

    def loop(seed, stream):
        gen = torch.Generator().manual_seed(seed)
        state, ch = prompt.PageState.allocate(B, 16, page, 48, DEV), prompt.Chunk.allocate(B, T, DEV)
        pk, pv = (torch.zeros(48, Hkv, page, D, dtype=BF, device=DEV) for _ in range(2))
        pages, ws = prompt.Pages(pk, pv, state.table), prompt.ChunkWorkspace(prob, T, DEV)
        x = [torch.randn(T, h, D, generator=gen).to(BF).to(DEV) for h in (Hq, Hkv, Hkv)]
        new = [i32(n) for n in ([120, 7, 150], [1, 1, 1], [90, 100, 1])]
        qo, out = (torch.zeros(T, Hq, D, dtype=BF, device=DEV) for _ in range(2))
        dense = hkv.Tier(*(torch.zeros(B, Hkv, 300, D, dtype=BF, device=DEV) for _ in range(2)), i32([0] * B * Hkv))
        head = i32([0] * B * Hkv)
        outs = [torch.zeros_like(out) for _ in new]
        torch.cuda.synchronize()

        def run():
            with torch.cuda.stream(stream):
                for n, o in zip(new, outs):
                    prompt.page_plan(ch.kv_len, n, state, state, ch, ws)
                    prompt.qk_norm_rope(prob, *x, ch.pos, rope, qo, ws, pages=pages, slot=ch.slot)
                    prompt.chunk_attention(prob, qo, ch.q_start, ch.kv_len, pages, o, ws)
                prompt.fill_tiers(prob, pages, ch.kv_len, dense, head, None, ws)
        return run, [*outs, pk, pv, dense.k, dense.v, dense.len, head, state.table], ws

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone = [loop(s, torch.cuda.current_stream()) for s in (26, 27)]
    for run, _, _ in alone:
        run()
        torch.cuda.synchronize()
    together = [loop(s, st) for s, st in zip((26, 27), streams)]
    for run, _, _ in together:
        run()
    torch.cuda.synchronize()
    for (_, a, wa), (_, b, wb) in zip(alone, together):
        assert wa.status() == 0 and wb.status() == 0
        for p, q in zip(a, b):
            assert torch.equal(p, q)


# one row tile whose key tiles go to both groups, one with a single key tile, two row tiles, and a mixture over many CTAs
KINDS = {"one": [(900, 1)], "short": [(20, 3)], "two": [(700, 200)], "all": [(900, 1), (20, 3), (700, 200), (5000, 90)] * 12}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", KINDS.values(), ids=KINDS)
def test_warps_give_up_as_one(lens, D):
    """Loads withheld, with limits from less than a poll of the clock to some hundred of them, so that lanes of a warp may
    see the limit pass at different polls: the kernel ends every time and the next call after a new start is right."""
    c = Case(lens, 8, 2, D, BF, 32, seed=29)
    for limit in (1, 3000, 50_000, 400_000):
        hkv.set_wait_limit_ns(limit)
        hkv.debug_withhold_publish(True)
        try:
            for _ in range(3):
                c.run()
            torch.cuda.synchronize()
        finally:
            hkv.debug_withhold_publish(False)
            hkv.set_wait_limit_ns(1_000_000_000)
        assert c.ws.status() == hkv.DEV_TIMEOUT
        c.ws.init()
    c.out.fill_(5.0), c.lse.fill_(5.0)
    c.run().check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", KINDS.values(), ids=KINDS)
def test_limits_that_pass_in_the_middle(lens, D):
    """Nothing is withheld, but the waits' limit is short, so that any of them may run out while loads and products are
    under way: the kernel lets them land and ends, the status word says so, or the results are right."""
    c = Case(lens, 8, 2, D, BF, 32, seed=30)
    ref = c.reference()
    c.reference = lambda: ref
    for limit in (1, 300, 1000, 3000, 10_000, 30_000, 100_000):
        hkv.set_wait_limit_ns(limit)
        try:
            c.out.fill_(5.0), c.lse.fill_(5.0)
            c.run()
            torch.cuda.synchronize()
        finally:
            hkv.set_wait_limit_ns(1_000_000_000)
        status = c.ws.status()
        assert status in (0, hkv.DEV_TIMEOUT)
        c.ws.init()
        if status == 0:
            c.check()
    c.out.fill_(5.0), c.lse.fill_(5.0)
    c.run().check()


@pytest.mark.parametrize("dtype,new", [(BF, 40), (F32, 40), (F32, 1)])
@pytest.mark.parametrize("where", ["behind", "between"])
def test_idle_requests_cost_a_scan_and_no_walk(dtype, new, where):
    """A table of 8192 slots with four requests in use, and the bits of a table of four. Every CTA scans the slots; it must
    not step over the idle ones one by one as well. At the end of the table nothing comes behind the four, so that call
    is the measure: with the four at the start it takes at most half as long again, with two at each end (a share then
    has 8188 idle slots in it, which a warp passes 32 at a time) at most 2.25 times as long. Step by step it was 11 to
    18 times in bf16 and 7 to 12 times in fp32."""
    B, Hq, Hkv, D, page = 8192, 8, 2, 64, 16
    # (rows for more than the slots' tokens: fp32 chunks run in the kernel for chunks)
    four = Case([(90, new), (300, new), (7, new), (150, new)], Hq, Hkv, D, dtype, page, pad=B if new > 1 else 0, seed=28).run()
    T = four.T

    def case(slots):
        table = torch.full((B, four.table.shape[1]), -1, dtype=torch.int32, device=DEV)
        n, kv = np.zeros(B, np.int32), np.full(B, 33, np.int32)
        for i, b in enumerate(slots):
            table[b], n[b], kv[b] = four.table[i], new, four.kv[i]
        prob = hkv.Problem(B, Hq, Hkv, D, dtype, 1.0, 0, 0)
        ws, out = prompt.ChunkWorkspace(prob, T, DEV), torch.full_like(four.out, 5.0)
        args = (prob, four.q, i32(np.concatenate([[0], np.cumsum(n)])), i32(kv), prompt.Pages(four.k, four.v, table), out, ws)
        prompt.chunk_attention(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                prompt.chunk_attention(*args)
        times = []
        for _ in range(8):
            a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            e.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(e) * 100)
        assert ws.status() == 0 and torch.equal(out, four.out)
        return min(times)

    last = case(range(B - 4, B))
    there = case(range(4) if where == "behind" else [0, 1, B - 2, B - 1])
    print(f"{dtype} {new} new: at the end {last:.1f} us, idle {where} {there:.1f} us")
    assert there <= 1.5 * last * (1.5 if where == "between" else 1.0)
