"""The prompt side's entry points: exported, refusing what they document as refused (nothing is launched, so no GPU
is used), and their oracle held to its own definitions."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import oracle
from oracle import prompt as op
from head_adaptive_kv_b200 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pr():
    hbuild.build()
    from head_adaptive_kv_b200 import prompt

    return prompt


@pytest.fixture(scope="module")
def hk(pr):
    from head_adaptive_kv_b200 import hkv

    return hkv


def test_every_declared_symbol_is_exported(pr):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hkv_prompt.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(hkv_[a-z_]+)\s*\(", text)))
    assert names == ["hkv_chunk_attention", "hkv_chunk_workspace_size", "hkv_fill_tiers", "hkv_page_plan",
                     "hkv_page_release", "hkv_qk_norm_rope"]
    for n in names:
        assert hasattr(pr.lib, n), n


def test_package_exports(pr):
    import head_adaptive_kv_b200 as pkg

    assert pkg.chunk_attention is pr.chunk_attention and pkg.Pages is pr.Pages


def _prob(hk, **kw):
    d = dict(B=2, Hq=8, Hkv=2, D=128, dtype=torch.bfloat16, p=0.9, bmin=4, bmax=64)
    d.update(kw)
    return hk.Problem(**d)


A = 0x10000  # aligned addresses that nothing reads


def _pages(pr, **kw):
    d = dict(k=A, v=2 * A, stride_p=2 * 16 * 128, stride_h=16 * 128, stride_t=128, pages=8, page=16, table=3 * A,
             table_stride=4, table_cols=4)
    d.update(kw)
    return pr._Pages(*[d[n] for n, _ in pr._Pages._fields_])


BAD_PAGES = {
    "page 24": dict(page=24), "page 8": dict(page=8), "page 512": dict(page=512), "page 0": dict(page=0),
    "negative pool": dict(pages=-1), "slots past 31 bits": dict(pages=1 << 27), "row stride": dict(table_stride=3),
    "table past 2^30 tokens": dict(table_stride=1 << 27, table_cols=(1 << 26) + 1), "no table": dict(table=None), "table alignment": dict(table=3 * A + 2),
}
BAD_STORAGE = {
    "no K": dict(k=None), "no V": dict(v=None), "K alignment": dict(k=A + 8), "token stride": dict(stride_t=64),
    "stride multiple": dict(stride_t=130), "head stride": dict(stride_h=-128),
}


def _plan(pr, B=2, ctx=A, new=A, pages=None, free=A, after_free=A, count=A, held=A, tokens=10, q_start=A, kv=A, pos=A,
          slot=A, granted=None, ws=A, nbytes=256):
    a, b = pr._State(free, count, held), pr._State(after_free, count, held)
    ch = pr._Chunk(tokens, q_start, kv, pos, slot)
    g = _pages(pr) if pages is None else pages
    return pr.lib.hkv_page_plan(B, ctx, new, C.byref(g), C.byref(a), C.byref(b), C.byref(ch), granted, ws, nbytes, None)


def test_page_plan_refusals(pr):
    for what, kw in BAD_PAGES.items():
        assert _plan(pr, pages=_pages(pr, **kw)) == 1, what
    for what, kw in {"B": dict(B=-1), "many": dict(B=8193), "ctx": dict(ctx=None), "new": dict(new=A + 2),
                     "free": dict(free=None, after_free=None), "two stacks": dict(after_free=2 * A),
                     "count": dict(count=None), "held": dict(held=None), "tokens": dict(tokens=(1 << 22) + 1),
                     "q_start": dict(q_start=None), "kv_len": dict(kv=None), "pos": dict(pos=None),
                     "slot": dict(slot=None), "granted": dict(granted=A + 1)}.items():
        assert _plan(pr, **kw) == 1, what
    for kw in (dict(ws=None), dict(ws=A + 16), dict(nbytes=128)):
        assert _plan(pr, **kw) == 6


def test_page_release_refusals(pr):
    s, g = pr._State(A, A, A), _pages(pr)
    call = lambda B=2, done=A, a=s, b=s, pages=g, ws=A: pr.lib.hkv_page_release(  # noqa: E731
        B, done, C.byref(pages), C.byref(a), C.byref(b), ws, 256, None)
    assert call(done=None) == 1 and call(B=-1) == 1 and call(B=8193) == 1
    assert call(a=pr._State(2 * A, A, A)) == 1 and call(pages=_pages(pr, page=20)) == 1
    assert call(ws=None) == 6


def _norm(pr, prob, q=A, k=2 * A, v=3 * A, qs=1024, ks=256, vs=256, T=5, pos=A, slot=None, rope=None, qw=A, kw=A, eps=1e-6,
          qo=4 * A, ko=5 * A, vo=6 * A, pages=None, ws=A):
    rope = pr._Rope(A, 128, 0, 1.0) if rope is None else rope
    return pr.lib.hkv_qk_norm_rope(C.byref(prob.c()), q, qs, k, ks, v, vs, T, pos, slot, C.byref(rope), qw, kw, eps, qo,
                                   ko, vo, None if pages is None else C.byref(pages), ws, 256, None)


def test_norm_rope_refusals(pr, hk):
    prob = _prob(hk)
    bad = {"q": dict(q=None), "q alignment": dict(q=A + 8), "k stride": dict(ks=128), "v stride": dict(vs=257),
           "tokens": dict(T=-1), "pos": dict(pos=None), "one weight": dict(kw=None), "eps": dict(eps=float("nan")),
           "negative eps": dict(eps=-1.0), "weights": dict(qw=A + 2, kw=A), "q_out": dict(qo=None),
           "k_out": dict(ko=None), "slot without pages": dict(slot=A), "rot": dict(rope=pr._Rope(A, 144, 0, 1.0)),
           "no angles": dict(rope=pr._Rope(None, 64, 0, 1.0)), "form": dict(rope=pr._Rope(A, 64, 2, 1.0)),
           "mscale": dict(rope=pr._Rope(A, 64, 0, float("nan")))}
    for what, kw in bad.items():
        assert _norm(pr, prob, **kw) == 1, what
    assert _norm(pr, prob, rope=pr._Rope(A, 40, 0, 1.0)) == 2
    assert _norm(pr, _prob(hk, D=96)) == 2
    paged = dict(pages=_pages(pr), ko=None, vo=None)
    assert _norm(pr, prob, **paged) == 1  # no slots
    assert _norm(pr, prob, pages=_pages(pr), slot=A) == 1  # and rows besides
    for what, kw in BAD_STORAGE.items():
        assert _norm(pr, prob, pages=_pages(pr, **kw), ko=None, vo=None, slot=A) == 1, what
    assert _norm(pr, prob, ws=None) == 6
    assert _norm(pr, prob, T=0) == 0  # nothing to do


def test_norm_rope_refuses_outputs_over_rows_that_others_still_read(pr, hk):
    """An output may stand on its own input, row on row; any other overlap would be written before it is read."""
    prob = _prob(hk)  # 8 query and 2 KV heads of 128 in bf16: rows of 2048 and 512 bytes
    far = 64 * A
    at = dict(q=A, k=2 * A, v=3 * A, qo=far, ko=2 * far, vo=3 * far)
    over = {"q in place, rows apart": dict(qo=A, qs=1536), "k in place, rows apart": dict(ko=2 * A, ks=512),
            "v in place, rows apart": dict(vo=3 * A, vs=264), "q_out a row into q": dict(qo=A + 2048),
            "q_out ends in k": dict(qo=2 * A - 5 * 2048 + 16), "k_out on v": dict(ko=3 * A),
            "v_out on k": dict(vo=2 * A), "k_out behind the first row of q": dict(ko=A + 2048),
            "q_out on k_out": dict(qo=2 * far), "k_out on v_out": dict(ko=3 * far),
            "v_out ends in q_out": dict(vo=far - 5 * 512 + 16),
            "slices of one projection, k_out on them": dict(q=A, k=A + 2048, v=A + 2560, qs=1536, ks=1536, vs=1536, ko=A + 4096)}
    for what, kw in over.items():
        assert _norm(pr, prob, **{**at, **kw}) == 1, what
    assert _norm(pr, prob, **{**at, "qo": A, "qs": 1536}, pages=_pages(pr), slot=A) == 1  # rows and pages besides
    paged = dict(at, ko=None, vo=None, pages=_pages(pr), slot=A)
    assert _norm(pr, prob, **{**paged, "qo": A, "qs": 1536}) == 1
    assert _norm(pr, prob, **{**paged, "qo": 3 * A}) == 1
    # what is allowed gets as far as the workspace: in place, one row of any stride, neighbours that touch
    allowed = [dict(), dict(qo=A), dict(qo=A, ko=2 * A, vo=3 * A), dict(T=1, qo=A, qs=1536, ko=2 * A, ks=512),
               dict(qo=A + 5 * 2048), dict(ko=2 * A - 5 * 512), dict(q=A, k=A + 2048, v=A + 2560, qs=1536, ks=1536, vs=1536)]
    for kw in allowed:
        assert _norm(pr, prob, ws=None, **{**at, **kw}) == 6, kw


def _attn(pr, prob, q=A, qs=1024, T=5, q_start=A, kv=A, pages=None, out=2 * A, lse=None, ws=A, nbytes=1 << 30):
    g = _pages(pr) if pages is None else pages
    return pr.lib.hkv_chunk_attention(C.byref(prob.c()), q, qs, T, q_start, kv, C.byref(g), out, lse, ws, nbytes, None)


def test_chunk_attention_refusals(pr, hk):
    prob = _prob(hk)
    for what, kw in {**BAD_PAGES, **BAD_STORAGE}.items():
        assert _attn(pr, prob, pages=_pages(pr, **kw)) == 1, what
    for what, kw in {"q": dict(q=None), "q alignment": dict(q=A + 8), "stride": dict(qs=512), "odd stride": dict(qs=1026),
                     "tokens": dict(T=-1), "many tokens": dict(T=(1 << 22) + 1), "q_start": dict(q_start=None),
                     "kv_len": dict(kv=None), "out": dict(out=None), "out alignment": dict(out=A + 4),
                     "lse": dict(lse=A + 2)}.items():
        assert _attn(pr, prob, **kw) == 1, what
    assert _attn(pr, _prob(hk, B=8193)) == 1
    assert _attn(pr, _prob(hk, Hq=6)) == 2 and _attn(pr, _prob(hk, D=256)) == 2
    assert _attn(pr, prob, ws=None) == 6 and _attn(pr, prob, ws=A + 8) == 6 and _attn(pr, prob, nbytes=256) == 6
    assert _attn(pr, prob, T=0) == 0 and _attn(pr, _prob(hk, B=0)) == 0


def test_chunk_attention_refuses_outputs_over_queries(pr, hk):
    """Other CTAs still read the queries when the first outputs are written: out and lse stand apart from q and from each
    other."""
    prob = _prob(hk)  # rows of 8 heads of 128 in bf16: 2048 bytes of q and out, 32 of lse
    at = dict(q=A, out=2 * A, lse=3 * A, T=5, nbytes=0)  # (what passes gets as far as the workspace)
    for what, kw in {"in place": dict(out=A), "a row further": dict(out=A + 2048), "up to the last row": dict(out=A + 8192),
                     "strided": dict(q=A, qs=1280, out=A + 4 * 2560 + 2032), "from before": dict(out=A - 5 * 2048 + 16),
                     "lse on q": dict(lse=A + 16), "lse on out": dict(lse=2 * A + 5 * 2048 - 4)}.items():
        assert _attn(pr, prob, **{**at, **kw}) == 1, what
    for what, kw in {"apart": dict(), "no lse": dict(lse=None), "behind": dict(out=A + 5 * 2048), "before": dict(out=A - 5 * 2048),
                     "strided": dict(qs=1280, out=A + 4 * 2560 + 2048), "lse behind": dict(lse=2 * A + 5 * 2048)}.items():
        assert _attn(pr, prob, **{**at, **kw}) == 6, what


def test_chunk_workspace_size(pr, hk):
    def size(T, **kw):
        n = C.c_size_t(0)
        code = pr.lib.hkv_chunk_workspace_size(C.byref(_prob(hk, **kw).c()), T, C.byref(n))
        return code, n.value

    code, one = size(1)
    assert code == 0 and one % 256 == 0
    assert size(1000)[1] > one and size(1 << 22)[1] == size(1000)[1]  # bounded: it does not grow with the prompt
    assert size(-1)[0] == 1 and size((1 << 22) + 1)[0] == 1 and size(1, D=96)[0] == 2


def test_fill_tiers_refusals(pr, hk):
    prob = _prob(hk)
    tier = lambda cap=8, k=A: hk._Tier(k, 2 * A, 2 * cap * 128, cap * 128, 128, cap, A)  # noqa: E731

    def call(pages=None, kv=A, take=None, dense=None, head=A, sparse=None, dropped=None, ws=A):
        g = _pages(pr) if pages is None else pages
        d, s = dense or tier(), sparse or tier()
        return pr.lib.hkv_fill_tiers(C.byref(prob.c()), C.byref(g), kv, take, C.byref(d), head, C.byref(s), dropped, ws,
                                     256, None)

    for what, kw in {**BAD_PAGES, **BAD_STORAGE}.items():
        assert call(pages=_pages(pr, **kw)) == 1, what
    assert call(kv=None) == 1 and call(head=None) == 1 and call(take=A + 1) == 1 and call(dropped=A + 2) == 1
    assert call(dense=tier(k=A + 8)) == 1 and call(sparse=tier(cap=-1)) == 1
    assert call(ws=None) == 6


def test_python_checks(pr, hk):
    """The binding's own checks, on CPU tensors (each raises before anything is called)."""
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    tab = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pr.Pages(k, k[:, :, :, :64].clone())
    with pytest.raises(ValueError):
        pr.Pages(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(TypeError):
        pr.Pages(k, k.clone(), tab.long())
    with pytest.raises(ValueError):
        pr.PageState(tab, torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                     torch.zeros(2, dtype=torch.int32), 16, 4)
    with pytest.raises(TypeError):
        pr.Rope(torch.zeros(32), 64)
    with pytest.raises(ValueError):
        pr.Rope(torch.zeros(16, dtype=torch.float64), 64)
    prob = _prob(hk)
    pages = pr.Pages(k, k.clone(), tab)
    with pytest.raises(TypeError):
        pages.fits(_prob(hk, dtype=torch.float32))
    with pytest.raises(ValueError):
        pages.fits(_prob(hk, B=3))
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        pr.chunk_attention(prob, q.float(), s, s[:2], pages, q, None)
    with pytest.raises(ValueError):
        pr.chunk_attention(prob, q, s[:2], s[:2], pages, torch.zeros_like(q), None)
    with pytest.raises(ValueError):
        pr.chunk_attention(prob, q[:, :, ::2], s, s[:2], pages, torch.zeros_like(q), None)
    rope = pr.Rope.of_base(128, 1e6, "cpu")
    assert rope.inv_freq.shape == (64,) and rope.inv_freq[0] == 1.0
    kv = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # neither pages nor rows
        pr.qk_norm_rope(prob, q, kv, kv, s, rope, torch.zeros_like(q), None)
    with pytest.raises(ValueError):  # both
        pr.qk_norm_rope(prob, q, kv, kv, s, rope, torch.zeros_like(q), None, k_out=kv, v_out=kv, pages=pages, slot=s)
    with pytest.raises(ValueError):
        pr.page_plan(s, s, pr.PageState.allocate(2, 2, 16, 4, "cpu"), None, None, None)


def test_oracle_attention_of_all_queries_is_causal_attention():
    """One request whose whole prompt is new: torch's own causal attention."""
    rng = np.random.default_rng(1)
    from tests.prompt_helpers import f64, pool

    k, v, table = pool(rng, 1, [37], 2, 64, 16, torch.float32)
    q = torch.randn(37, 4, 64)
    out, lse, *_ = op.chunk_attention(f64(q), f64(k), f64(v), [0, 37], [37], table.numpy(), 16, 0.125)
    ids = table[0].long()
    kk, vv = (x[ids].transpose(0, 1).reshape(2, -1, 64)[:, :37].double().repeat_interleave(2, 0) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1)[None], kk[None], vv[None],
                                                            is_causal=True, scale=0.125)[0].transpose(0, 1)
    assert np.abs(out - want.numpy()).max() < 1e-12
    assert np.isfinite(lse).all()


def test_oracle_norm_rope_keeps_lengths_and_turns_by_position():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 2, 64)), np.ones(64)
    f = 10000.0 ** (-np.arange(16) / 16)
    y, _ = op.norm_rope(x, w, np.array([0, 5, 9]), f, 32, False, 1.0, 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    assert np.allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True)))
    # the product of two turned rows depends on the distance of their positions only
    a, _ = op.norm_rope(np.tile(x[:1], (2, 1, 1)), None, np.array([3, 103]), f, 32, True, 1.0, 0.0)
    b, _ = op.norm_rope(np.tile(x[1:2], (2, 1, 1)), None, np.array([7, 107]), f, 32, True, 1.0, 0.0)
    d = (a * b).sum(-1)
    assert np.allclose(d[0], d[1])


def test_oracle_plan_and_release_keep_every_page_once():
    rng = np.random.default_rng(3)
    B, page, pages, cols = 6, 16, 40, 12
    table = np.full((B, cols), -1, np.int32)
    free, count, held = np.arange(pages, dtype=np.int32)[::-1].copy(), pages, np.zeros(B, np.int32)
    ctx = np.zeros(B, np.int32)
    for step in range(30):
        new = rng.integers(0, 40, B).astype(np.int32)
        r = op.plan(ctx, new, held, free, count, table, page, 100)
        table, held, count, ctx = r["table"], r["held"], r["count"], r["kv_len"]
        used = [p for b in range(B) for p in table[b, :held[b]]]
        assert sorted(used + list(free[:count])) == list(range(pages))
        assert len(set(r["slot"][r["slot"] >= 0].tolist())) == int(r["granted"].sum())
        done = (rng.random(B) < 0.3).astype(np.int32)
        free, count, held = op.release(done, held, free, count, table)
        ctx = np.where(done, 0, ctx)


def test_oracle_fill_without_a_window_is_the_prompt_itself():
    rng = np.random.default_rng(4)
    from tests.prompt_helpers import pool

    k, v, table = pool(rng, 1, [20], 1, 64, 16, torch.float32)
    z = lambda n: np.zeros((1, 1, n, 64), np.float32)  # noqa: E731
    i = np.zeros(1, np.int32)
    d, h, s, lost = op.fill(k.numpy(), v.numpy(), table.numpy(), 16, [20], oracle.Tier(z(0), z(0), i), i,
                            oracle.Tier(z(18), z(18), i))
    rows = k[table[0].long()].transpose(0, 1).reshape(1, -1, 64)[:, :18]
    assert np.array_equal(s.k[0], rows.numpy()) and s.len[0] == 18 and lost[0] == 2 and h[0] == 0
