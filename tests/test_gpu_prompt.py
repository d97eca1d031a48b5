"""GPU parity of the page plan, the norms with rotation and the tier fill against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from head_adaptive_kv_b200 import hkv, prompt
from head_adaptive_kv_b200.workloads import to_host_bits
from oracle import prompt as op
from tests.prompt_helpers import f64, norm_bounds, pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


# ---- page plan and release ----------------------------------------------------


def run_plan(ctx, new, held, free, count, table, page, T, in_place=False):
    st = prompt.PageState(i32(table), i32(free), i32([count]), i32(held), page, len(free))
    after = st if in_place else prompt.PageState(st.table, st.free, i32([-7]), i32([-7] * len(held)), page, len(free))
    ch = prompt.Chunk.allocate(len(held), T, DEV)
    ch.pos.fill_(77), ch.slot.fill_(77)
    ws = prompt.status_workspace(DEV)
    granted = i32([-7] * len(held))
    prompt.page_plan(i32(ctx), i32(new), st, after, ch, ws, granted=granted)
    return st, after, ch, granted, ws.status()


def check_plan(ctx, new, held, free, count, table, page, T, in_place=False):
    ref = op.plan(ctx, new, held, free, count, table, page, T)
    st, after, ch, granted, status = run_plan(ctx, new, held, free, count, table, page, T, in_place)
    for got, name in ((st.table, "table"), (after.held, "held"), (ch.q_start, "q_start"), (ch.kv_len, "kv_len"),
                      (ch.pos, "pos"), (ch.slot, "slot"), (granted, "granted")):
        assert np.array_equal(got.cpu().numpy(), ref[name]), name
    assert int(after.free_count) == ref["count"]
    assert np.array_equal(st.free.cpu().numpy(), free)
    nowhere = ((ref["pos"] >= 0) & (ref["slot"] < 0)).any()  # a table entry that is no page of the pool
    assert status == (prompt.DEV_PAGES_FULL if ref["left"] else 0) | (hkv.DEV_BAD_INDEX if ref["bad"] or nowhere else 0)
    return ref


def state(rng, B, page, ctx, spare, cols=None):
    ctx = np.asarray(ctx)
    held = -(-ctx // page)
    total = int(held.sum()) + spare
    ids = rng.permutation(total).astype(np.int32)
    cols = int(held.max(initial=0)) + 6 if cols is None else cols
    table, at = np.full((B, cols), -1, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(total, -1, np.int32)
    free[:spare] = ids[at:]
    return held.astype(np.int32), free, spare, table


@pytest.mark.parametrize("B,page,hi,T", [(1, 16, 1, 1), (3, 16, 40, 100), (64, 64, 5, 200), (513, 32, 3, 2000),
                                         (1025, 16, 2, 700), (200, 256, 300, 40000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, page, hi, T, in_place):
    rng = np.random.default_rng(B + page)
    ctx, new = rng.integers(0, 300, B), rng.integers(0, hi + 1, B)
    held, free, count, table = state(rng, B, page, ctx, 4 * B + 3, cols=300 // page + hi // page + 3)
    check_plan(ctx, new, held, free, count, table, page, T, in_place)


def test_plan_edges():
    rng = np.random.default_rng(5)
    z = np.zeros(4, np.int64)
    # nothing cached, one token each; a whole page to the last row; nothing to do at all
    for new in ([1, 1, 1, 1], [16, 17, 15, 32], [0, 0, 0, 0]):
        held, free, count, table = state(rng, 4, 16, z, 12)
        check_plan(z, new, held, free, count, table, 16, sum(new))
    # the last row of a page, and the first of the next
    ctx = np.array([15, 16, 31, 32])
    held, free, count, table = state(rng, 4, 16, ctx, 4)
    check_plan(ctx, [1, 1, 1, 1], held, free, count, table, 16, 9)
    # pages held ahead of need are used up first
    held, free, count, table = state(rng, 4, 16, np.array([40, 40, 40, 40]), 4)
    check_plan([3, 20, 0, 40], [30, 20, 48, 8], held, free, count, table, 16, 200)


def test_plan_without_room():
    rng = np.random.default_rng(6)
    ctx = np.array([10, 0, 5, 16, 7])
    for spare, T in ((2, 400), (3, 400), (0, 400), (100, 60), (100, 0), (100, 41)):
        held, free, count, table = state(rng, 5, 16, ctx, spare, cols=8)
        ref = check_plan(ctx, [20, 21, 3, 16, 1], held, free, count, table, 16, T)
        assert ref["left"]


def test_plan_of_bad_requests_leaves_them_out():
    rng = np.random.default_rng(7)
    ctx = np.array([10, 0, 5, 16, 7, 3, 1])
    held, free, count, table = state(rng, 7, 16, ctx, 30, cols=4)
    bad_ctx, new = np.array([10, -1, 5, 40, 7, 3, 2**31 - 1]), np.array([1, 1, -5, 1, 60, 4, 2**31 - 1])
    ref = check_plan(bad_ctx, new, held, free, count, table, 16, 100)
    assert ref["bad"] == [1, 2, 3, 4, 6]
    held[5] = 9  # more than the table has
    assert check_plan(ctx, [1] * 7, held, free, count, table, 16, 100)["bad"] == [5]


def test_plan_with_a_bad_count_or_bad_pages():
    rng = np.random.default_rng(8)
    ctx = np.array([16, 15])
    held, free, count, table = state(rng, 2, 16, ctx, 3)
    st, after, ch, granted, status = run_plan(ctx, [1, 1], held, free, 99, table, 16, 4)
    assert status == prompt.DEV_PAGES_FULL | hkv.DEV_BAD_INDEX
    assert granted.tolist() == [0, 1] and int(after.free_count) == 99  # only the request that needs no page
    free[count - 1], table[1, 0] = 1000, -3
    st, after, ch, granted, status = run_plan(ctx, [1, 1], held, free, count, table, 16, 4)
    assert status == hkv.DEV_BAD_INDEX
    assert ch.slot.tolist() == [-1] * 4 and ch.pos.tolist() == [16, 15, -1, -1]


def test_release_and_plan_over_many_steps():
    rng = np.random.default_rng(9)
    B, page, pages, cols, T = 37, 16, 300, 20, 700
    st = prompt.PageState.allocate(B, cols, page, pages, DEV)
    ch, ws = prompt.Chunk.allocate(B, T, DEV), prompt.status_workspace(DEV)
    table, free = st.table.cpu().numpy(), st.free.cpu().numpy()
    count, held, ctx = pages, np.zeros(B, np.int32), np.zeros(B, np.int32)
    dctx = i32(ctx)
    for _ in range(12):
        new, done = rng.integers(0, 60, B), (rng.random(B) < 0.25).astype(np.int32)
        prompt.page_release(i32(done), st, st, ws)
        free, count, held = op.release(done, held, free, count, table)
        ctx = np.where(done, 0, ctx)
        dctx = torch.where(i32(done) != 0, 0, dctx).to(torch.int32)
        prompt.page_plan(dctx, i32(new), st, st, ch, ws)
        r = op.plan(ctx, new, held, free, count, table, page, T)
        table, held, count, ctx = r["table"], r["held"], r["count"], r["kv_len"]
        dctx = ch.kv_len.clone()
        assert ws.status() == (prompt.DEV_PAGES_FULL if r["left"] else 0) | (hkv.DEV_BAD_INDEX if r["bad"] else 0)
        for got, want in ((st.table, table), (st.free, free), (st.held, held), (ch.slot, r["slot"]), (ch.kv_len, ctx)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(st.free_count) == count


def test_plan_advances_lengths_in_place():
    """ctx_len and kv_len one tensor: each call's lengths are the next one's."""
    B, page = 700, 16  # more requests than the scan's strip
    st, ch = prompt.PageState.allocate(B, 4, page, 4 * B, DEV), prompt.Chunk.allocate(B, 3 * B, DEV)
    ws = prompt.status_workspace(DEV)
    ctx = np.zeros(B, np.int32)
    held, free, count, table = ctx.copy(), st.free.cpu().numpy(), 4 * B, st.table.cpu().numpy()
    for step in range(6):
        new = (np.arange(B) + step) % 5
        prompt.page_plan(ch.kv_len, i32(new), st, st, ch, ws)
        r = op.plan(ctx, new, held, free, count, table, page, 3 * B)
        ctx, held, count, table = r["kv_len"], r["held"], r["count"], r["table"]
        assert np.array_equal(ch.kv_len.cpu().numpy(), ctx) and np.array_equal(ch.slot.cpu().numpy(), r["slot"])
        assert np.array_equal(st.table.cpu().numpy(), table) and int(st.free_count) == count
    assert ws.status() == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_and_release_of_the_most_requests(in_place):
    """8192 requests, the limit of a call: sixteen strips of the scan, the whole of its shared memory."""
    B, page = 8192, 16
    rng = np.random.default_rng(12)
    ctx, new = rng.integers(0, 100, B), rng.integers(0, 4, B)
    held, free, count, table = state(rng, B, page, ctx, B // 2)
    ref = check_plan(ctx, new, held, free, count, table, page, 2 * B, in_place)
    assert not ref["left"] and not ref["bad"] and ref["q_start"][-1] == new.sum() > B  # 1.5 tokens a request
    done = (rng.random(B) < 0.5).astype(np.int32)
    st = prompt.PageState(i32(ref["table"]), i32(free), i32([ref["count"]]), i32(ref["held"]), page, len(free))
    ws = prompt.status_workspace(DEV)
    prompt.page_release(i32(done), st, st, ws)
    stack, top, kept = op.release(done, ref["held"], free, ref["count"], ref["table"])
    assert ws.status() == 0 and int(st.free_count) == top
    assert np.array_equal(st.free.cpu().numpy(), stack) and np.array_equal(st.held.cpu().numpy(), kept)


def test_release_of_a_state_that_does_not_fit():
    st = prompt.PageState.allocate(3, 4, 16, 10, DEV)
    ws = prompt.status_workspace(DEV)
    for held, count in (([1, 5, 0], 0), ([1, -1, 0], 0), ([4, 4, 0], 3), ([1, 1, 1], -2)):
        st.held.copy_(i32(held))
        st.free_count.copy_(i32([count]))
        free = st.free.clone()
        prompt.page_release(i32([1, 1, 0]), st, st, ws)
        assert ws.status() == hkv.DEV_BAD_INDEX
        assert st.held.tolist() == held and st.free_count.tolist() == [count] and torch.equal(st.free, free)


@pytest.mark.parametrize("B", [3, 200])  # one CTA's share of the requests, and several
@pytest.mark.parametrize("entry", [-1, -2**31, 2**31 - 1, "pages"])
def test_release_of_entries_that_are_no_pages(B, entry):
    """A table entry that names no page of the pool must not reach the stack, where it would be given out again: the
    whole release is refused, and one without the request that holds the entry goes through."""
    page, cols = 16, 3
    st = prompt.PageState.allocate(B, cols, page, B * cols, DEV)
    ws, ch = prompt.status_workspace(DEV), prompt.Chunk.allocate(B, B * cols * page, DEV)
    prompt.page_plan(i32([0] * B), i32([cols * page] * B), st, st, ch, ws)
    assert ws.status() == 0 and int(st.free_count) == 0
    bad = B - 2  # its last column, as far as a page number goes
    st.table[bad, cols - 1] = B * cols if entry == "pages" else entry
    st.free.fill_(-9)
    before = [x.clone() for x in (st.table, st.free, st.free_count, st.held)]
    after = prompt.PageState(st.table, st.free, i32([-7]), i32([-7] * B), page, B * cols)
    prompt.page_release(i32([1] * B), st, after, ws)
    assert ws.status() == hkv.DEV_BAD_INDEX
    assert int(after.free_count) == 0 and after.held.tolist() == [cols] * B
    for x, y in zip((st.table, st.free, st.free_count, st.held), before):
        assert torch.equal(x, y)
    done = np.ones(B, np.int32)
    done[bad] = 0
    free, count, held = op.release(done, st.held.cpu().numpy(), st.free.cpu().numpy(), 0, st.table.cpu().numpy())
    prompt.page_release(i32(done), st, st, ws)
    assert ws.status() == 0 and int(st.free_count) == count
    assert np.array_equal(st.free.cpu().numpy(), free) and np.array_equal(st.held.cpu().numpy(), held)


# ---- norms and rotation ---------------------------------------------------------


def norm_case(T, Hq, Hkv, D, dtype, rot, inter=False, norm=True, seed=0, far=False):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * 3).to(dtype).to(DEV)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).to(DEV) if norm else None for _ in range(2)]
    pos = torch.randint(0, 2**31 - 1 if far else 5000, (T,), generator=g).to(torch.int32).to(DEV)
    rope = prompt.Rope.of_base(rot, 1e6, DEV, inter) if rot else prompt.Rope(None, 0)
    return qkv, q, k, v, w, pos, rope, hkv.Problem(1, Hq, Hkv, D, dtype, 1.0, 0, 0)


def norm_ref(q, k, w, pos, rope, inter, mscale=1.0):
    f = f64(rope.inv_freq) if rope.rot else np.zeros(0)
    return [op.norm_rope(f64(x), None if y is None else f64(y), pos.cpu().numpy(), f, rope.rot, inter, mscale, 1e-6)
            for x, y in zip((q, k), w)]


CASES = [  # T, Hq, Hkv, D, dtype, rot, interleaved, norm, far positions
    (1, 1, 1, 64, torch.bfloat16, 64, False, True, False),
    (7, 32, 8, 128, torch.bfloat16, 128, False, True, False),
    (601, 8, 2, 128, torch.bfloat16, 128, False, True, True),
    (33, 8, 1, 64, torch.bfloat16, 32, True, True, False),
    (5, 2, 2, 128, torch.bfloat16, 96, False, False, False),
    (9, 4, 2, 128, torch.bfloat16, 0, False, True, False),
    (1000, 4, 2, 64, torch.float32, 64, False, True, True),
    (31, 16, 2, 128, torch.float32, 48, True, True, False),
    (3, 3 * 4, 3, 128, torch.float32, 16, False, True, False),
    (593, 1, 1, 64, torch.float32, 16, True, False, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("to_pages", [False, True])
def test_norm_rope(case, to_pages):
    T, Hq, Hkv, D, dtype, rot, inter, norm, far = case
    qkv, q, k, v, w, pos, rope, prob = norm_case(T, Hq, Hkv, D, dtype, rot, inter, norm, T, far)
    before = qkv.clone()
    skip = torch.arange(T, device=DEV) % 5 == 3  # rows behind or between the tokens
    pos = torch.where(skip, -1, pos).to(torch.int32)
    qo = torch.full((T, Hq, D), 7.0, dtype=dtype, device=DEV)
    ws = prompt.status_workspace(DEV)
    kw = dict(q_weight=w[0], k_weight=w[1])
    if to_pages:
        rng = np.random.default_rng(T)
        page = 16
        P = T // page + 2
        slots = i32(rng.permutation(P * page)[:T])
        slots[::7] = -1
        store = [torch.full((P, page, Hkv, D + 8), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
        kp, vp = (x[..., :D].transpose(1, 2) for x in store)
        prompt.qk_norm_rope(prob, q, k, v, pos, rope, qo, ws, pages=prompt.Pages(kp, vp), slot=slots, **kw)
        at = slots.long()
        ko, vo = (x[at.clamp(min=0) // page, :, at.clamp(min=0) % page] for x in (kp, vp))
        written = ~skip & (slots >= 0)
        rest = torch.ones(P * page, dtype=torch.bool, device=DEV)
        rest[at[written]] = False
        for x in store:  # nothing but the tokens' rows is touched
            assert (x.view(P * page, Hkv, D + 8)[rest] == 7.0).all() and (x[..., D:] == 7.0).all()
    else:
        ko, vo = (torch.full((T, Hkv, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        prompt.qk_norm_rope(prob, q, k, v, pos, rope, qo, ws, k_out=ko, v_out=vo, **kw)
        written = ~skip
        assert (ko[skip] == 7.0).all() and (vo[skip] == 7.0).all()
    assert ws.status() == 0
    assert torch.equal(qkv, before)
    assert (qo[skip] == 7.0).all()
    assert torch.equal(vo[written], v[written])
    for got, (ref, mag), rows in zip((qo, ko), norm_ref(q, k, w, pos.clamp(min=0), rope, inter), (~skip, written)):
        r = rows.cpu().numpy()
        err = np.abs(f64(got) - ref)[r]
        assert (err <= norm_bounds(ref, mag, dtype == torch.bfloat16)[r]).all(), err.max()


def test_norm_rope_in_place_and_mscale():
    qkv, q, k, v, w, pos, rope, prob = norm_case(20, 8, 2, 128, torch.bfloat16, 128)
    rope = prompt.Rope(rope.inv_freq, 128, False, 0.75)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    refs = norm_ref(q, k, w, pos, rope, False, 0.75)
    v0 = v.clone()
    ws = prompt.status_workspace(DEV)
    prompt.qk_norm_rope(prob, q, k, v, pos, rope, q, ws, q_weight=w[0], k_weight=w[1], k_out=k, v_out=v)
    assert torch.equal(v, v0)
    for got, (ref, mag) in zip((q, k), refs):
        assert (np.abs(f64(got) - ref) <= norm_bounds(ref, mag, True)).all()


def test_norm_rope_bad_slots_are_reported_and_not_written():
    qkv, q, k, v, w, pos, rope, prob = norm_case(4, 4, 2, 64, torch.float32, 64)
    kp, vp = (torch.zeros(2, 2, 16, 64, device=DEV) for _ in range(2))
    qo, ws = torch.zeros(4, 4, 64, device=DEV), prompt.status_workspace(DEV)
    for slots, bad in (([32, -1, 3, 2], True), ([-2, 4, 5, 6], True), ([2**31 - 1, 1, 2, 3], True), ([0, -1, 31, 2], False)):
        kp.zero_(), vp.zero_()
        prompt.qk_norm_rope(prob, q, k, v, pos, rope, qo, ws, q_weight=w[0], k_weight=w[1], pages=prompt.Pages(kp, vp),
                            slot=i32(slots))
        assert ws.status() == (hkv.DEV_BAD_INDEX if bad else 0)
        good = [s for s in slots if 0 <= s < 32]
        touched = (vp.transpose(1, 2).reshape(32, -1) != 0).any(1).nonzero().flatten().tolist()
        assert touched == sorted(good)


def test_norm_rope_of_zero_rows_and_of_zeros():
    qkv, q, k, v, w, pos, rope, prob = norm_case(3, 4, 2, 64, torch.bfloat16, 64)
    ws = prompt.status_workspace(DEV)
    z = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    zk = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    prompt.qk_norm_rope(prob, z, zk, zk, pos[:0], rope, z, ws, k_out=zk, v_out=zk)
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    qo, ko, vo = torch.ones_like(q), torch.ones_like(k), torch.ones_like(k)
    prompt.qk_norm_rope(prob, q, k, v, pos, rope, qo, ws, q_weight=w[0], k_weight=w[1], k_out=ko, v_out=vo)
    assert (qo == 0).all() and (ko == 0).all() and ws.status() == 0


# ---- tiers from pages ------------------------------------------------------------


@pytest.mark.parametrize("dtype,D,page,layout", [(torch.bfloat16, 128, 16, "hnd"), (torch.bfloat16, 64, 64, "nhd"),
                                                 (torch.float32, 128, 32, "nhd"), (torch.float32, 64, 256, "hnd")])
@pytest.mark.parametrize("wcap,ncap", [(16, 200), (1, 50), (64, 100), (0, 150), (40, 0), (500, 500)])
def test_fill_tiers(dtype, D, page, layout, wcap, ncap):
    rng = np.random.default_rng(wcap + ncap + D)
    lens, Hkv = [0, 1, 16, 17, 64, 65, 141, 300], 2
    B = len(lens)
    take = np.array([1, 1, 1, 1, 1, 0, 1, 1], np.int32)
    k, v, table = pool(rng, B, lens, Hkv, D, page, dtype, layout=layout, device=DEV)
    prob = hkv.Problem(B, Hkv, Hkv, D, dtype, 1.0, 0, 0)
    g = torch.Generator().manual_seed(3)

    def tier(cap):  # rows 8 elements apart, old contents in all of it
        a, b = (torch.randn(B, Hkv, cap, D + 8, generator=g).to(dtype).to(DEV) for _ in range(2))
        return a, b, hkv.Tier(a[..., :D], b[..., :D], i32(rng.integers(0, cap + 1, B * Hkv)))

    (da, db, dense), (sa, sb, sparse) = tier(wcap), tier(ncap)
    head, dropped = i32([3] * B * Hkv), i32([-1] * B * Hkv)
    host = lambda t: oracle.Tier(to_host_bits(t.k), to_host_bits(t.v), t.len.cpu().numpy().copy())  # noqa: E731
    d, h, s, lost = op.fill(to_host_bits(k), to_host_bits(v), table.cpu().numpy(), page, lens, host(dense),
                            head.cpu().numpy(), host(sparse), take)
    pads = [x[..., D:].clone() for x in (da, db, sa, sb)]
    ws = prompt.status_workspace(DEV)
    prompt.fill_tiers(prob, prompt.Pages(k, v, table), i32(lens), dense if wcap else None, head if wcap else None,
                      sparse if ncap else None, ws, take=i32(take), dropped=dropped)
    assert ws.status() == (hkv.DEV_SPARSE_FULL if lost.any() else 0)
    taken = np.repeat(take, Hkv) != 0
    if wcap:
        for got, want in ((host(dense).k, d.k), (host(dense).v, d.v), (host(dense).len, d.len), (head.cpu().numpy(), h)):
            assert np.array_equal(got, want)
    if ncap:
        for got, want in ((host(sparse).k, s.k), (host(sparse).v, s.v), (host(sparse).len, s.len)):
            assert np.array_equal(got, want)
    assert np.array_equal(dropped.cpu().numpy()[taken], lost[taken]) and (dropped.cpu().numpy()[~taken] == -1).all()
    for x, old in zip((da, db, sa, sb), pads):
        assert torch.equal(x[..., D:], old)


def test_fill_tiers_of_bad_lengths_and_pages():
    rng = np.random.default_rng(1)
    k, v, table = pool(rng, 2, [40, 40], 1, 64, 16, torch.float32, device=DEV)
    prob, ws = hkv.Problem(2, 1, 1, 64, torch.float32, 1.0, 0, 0), prompt.status_workspace(DEV)
    make = lambda n: hkv.Tier(torch.ones(2, 1, n, 64, device=DEV), torch.ones(2, 1, n, 64, device=DEV), i32([0, 0]))  # noqa: E731
    dense, sparse, head = make(8), make(64), i32([0, 0])
    table[1, 1] = 999
    prompt.fill_tiers(prob, prompt.Pages(k, v, table), i32([-4, 40]), dense, head, sparse, ws)
    assert ws.status() == hkv.DEV_LEN_CLAMPED | hkv.DEV_BAD_INDEX
    assert dense.len.tolist() == [0, 8] and sparse.len.tolist() == [0, 32]
    assert (sparse.k[1, 0, 16:32] == 0).all() and torch.equal(sparse.k[1, 0, :16], k[int(table[1, 0]), 0])
    table[1, 1] = 0
    prompt.fill_tiers(prob, prompt.Pages(k, v, table), i32([40, 1 << 30]), dense, head, sparse, ws)
    assert ws.status() == hkv.DEV_LEN_CLAMPED and dense.len.tolist() == [8, 8] and sparse.len.tolist() == [32, 40]
