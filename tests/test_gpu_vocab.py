"""The embedding lookup and its gradient, and the head's cross entropy and its
gradient, against 64-bit formulas on the CPU within the bounds their roundings
allow (vocab_util)."""
import numpy as np
import pytest
import torch

import vocab_util as vu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import trie_constrained_beam_step_amd as gr
    return gr


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _tokens(n, vocab, gen, hot=0.0, absent=0.15):
    """Random tokens; a share of them one hot word, a share outside [0, vocab)."""
    t = torch.randint(0, vocab, (n,), generator=gen)
    t = torch.where(torch.rand(n, generator=gen) < hot, vocab // 3, t)
    bad = torch.tensor([-1, vocab, -(2 ** 31), 2 ** 31 - 1])[torch.randint(0, 4, (n,), generator=gen)]
    return torch.where(torch.rand(n, generator=gen) < absent, bad, t).to(torch.int32)


def _strided(x, pad, off):
    """x on the GPU in rows `pad` elements further apart, `off` elements into a
    buffer of NaN (what a kernel must not read shows up)."""
    n, d = x.shape
    buf = torch.full((off + n * (d + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[off:off + n * (d + pad)].view(n, d + pad)[:, :d]
    v.copy_(x)
    return v


def _guarded(n, d, dtype, pad=0, off=0):
    """An output of n rows inside a buffer of a known value, and a check that
    nothing outside the rows was written."""
    buf = torch.full((off + n * (d + pad) + 64,), 7.0, dtype=dtype, device="cuda")
    body = buf[off:off + n * (d + pad)].view(n, d + pad)

    def untouched():
        assert bool((buf[:off] == 7).all()) and bool((buf[off + n * (d + pad):] == 7).all())
        assert bool((body[:, d:] == 7).all())
    return body[:, :d], untouched


# ---------------------------------------------------------------- embedding

LOOKUPS = [(1, 48, 64), (16, 48, 64), (5, 1, 1), (33, 7, 3), (257, 1280, 100), (1000, 50_257, 67), (64, 300, 1024),
           (3, 20, 4100)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", LOOKUPS)
def test_lookup(gr, dtype, n, vocab, dim):
    gen = _gen(n * 7 + dim)
    w = torch.randn(vocab, dim, generator=gen).to(vu.DT[dtype])
    t = _tokens(n, vocab, gen)
    e = gr.Embedding(vocab, dim, max_tokens=n, dtype=dtype, scale=1.7)
    ok = ((t >= 0) & (t < vocab))[:, None]
    scale = float(np.float32(1.7))
    want = torch.where(ok, w[t.clamp(0, vocab - 1).long()].float() * scale, 0.0).to(vu.DT[dtype])
    assert torch.equal(e.lookup(t.cuda(), w.cuda()).cpu(), want)
    for pad, off in ((1, 1), (8, 8)):
        out, untouched = _guarded(n, dim, vu.DT[dtype], pad, off)
        e.lookup(t.cuda(), _strided(w, pad, off), out=out)
        assert torch.equal(out.cpu(), want)
        untouched()
    e.close()


# the last: enough hot tokens to split a word's rows
SCATTERS = [(1, 48, 64, 0.0), (48, 48, 64, 0.5), (5, 1, 1, 0.0), (300, 7, 3, 0.3), (1000, 1280, 100, 0.4),
            (2049, 50_257, 67, 0.1), (4096, 300, 256, 0.0), (5000, 5, 130, 0.9), (70_000, 1000, 33, 0.6)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim,hot", SCATTERS)
def test_embedding_gradient(gr, dtype, n, vocab, dim, hot):
    gen = _gen(n * 5 + dim)
    t = _tokens(n, vocab, gen, hot)
    g = torch.randn(n, dim, generator=gen).to(vu.DT[dtype])
    ok = (t >= 0) & (t < vocab)
    g[~ok] = float("nan")  # rows of absent tokens are not used
    base = torch.randn(vocab, dim, generator=gen).to(vu.DT[dtype])
    e = gr.Embedding(vocab, dim, max_tokens=n + 3, dtype=dtype, scale=-0.75)
    want, err = vu.scatter(t, torch.where(ok[:, None], g, 0), vocab, -0.75, dtype)
    first = e.backward(t.cuda(), g.cuda())
    vu.check("grad_weight", first, want, err)
    assert torch.equal(first, e.backward(t.cuda(), g.cuda())), "two calls differ"
    want, err = vu.scatter(t, torch.where(ok[:, None], g, 0), vocab, -0.75, dtype, base)
    for pad, off in ((0, 0), (1, 1), (8, 8)):
        out, untouched = _guarded(vocab, dim, vu.DT[dtype], pad, off)
        out.copy_(base)
        e.backward(t.cuda(), _strided(g, pad, off), grad_weight=out, accumulate=True)
        vu.check("accumulated grad_weight", out, want, err)
        untouched()
    e.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [[], [-1, -1, 99], [4] * 500])
def test_embedding_gradient_without_rows(gr, dtype, tokens):
    """No tokens, none inside the table, and one word alone."""
    t = torch.tensor(tokens, dtype=torch.int32)
    g = torch.randn(len(tokens), 40, generator=_gen(1)).to(vu.DT[dtype])
    e = gr.Embedding(99, 40, max_tokens=512, dtype=dtype)
    want, err = vu.scatter(t, g, 99, 1.0, dtype)
    vu.check("grad_weight", e.backward(t.cuda(), g.cuda()), want, err)
    base = torch.randn(99, 40, generator=_gen(2)).to(vu.DT[dtype])
    out = base.cuda()
    e.backward(t.cuda(), g.cuda(), grad_weight=out, accumulate=True)
    want, err = vu.scatter(t, g, 99, 1.0, dtype, base)
    vu.check("accumulated grad_weight", out, want, err)
    assert e.lookup(t.cuda(), base.cuda()).shape == (len(tokens), 40)
    e.close()


# --------------------------------------------------------------------- head

HEADS = [(1, 48, 64), (48, 48, 64), (1, 1, 1), (3, 5, 7), (17, 1280, 96), (16, 513, 128), (33, 300, 1000),
         (65, 1000, 67), (130, 257, 256), (300, 770, 200), (700, 130, 64), (257, 2100, 130),
         (4096, 64, 512), (4097, 64, 512), (9, 512, 64), (200, 449, 63), (35, 15, 256), (64, 256, 64), (65, 257, 64)]


def _head_inputs(n, vocab, dim, dtype, seed, absent=0.2):
    gen = _gen(seed)
    t = _tokens(n, vocab, gen, 0.2, absent if n > 1 else 0.0)
    ok = (t >= 0) & (t < vocab)
    w = (torch.randn(vocab, dim, generator=gen) * (1.5 * dim ** -0.5)).to(vu.DT[dtype])
    h = torch.randn(n, dim, generator=gen)
    h = (h + 4 * torch.rand(n, 1, generator=gen) * w[t.clamp(0, vocab - 1).long()].float()).to(vu.DT[dtype])
    g = torch.randn(n, generator=gen) * 0.1
    clean = h.clone(), g.clone()
    h[~ok] = float("nan")
    g[~ok] = float("inf")
    return h, w, t, g, clean


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", HEADS)
def test_head(gr, dtype, n, vocab, dim):
    h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, dtype, n + vocab)
    base = torch.randn(vocab, dim, generator=_gen(9)).to(vu.DT[dtype])
    scale = 1.25
    want = vu.head(hc, w, t, scale, dtype, gc)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype, scale=scale)
    tc, gcu = t.cuda(), g.cuda()
    for pad, off in ((0, 0), (1, 1), (8, 8)):
        hs, ws = _strided(h, pad, off), _strided(w, pad, off)
        loss, lse = head.loss(hs, ws, tc)
        vu.check("loss", loss, want["loss"], want["loss_err"])
        vu.check("lse", lse, want["lse"], want["lse_err"])
        gh, ghu = _guarded(n, dim, vu.DT[dtype], pad, off)
        gw, gwu = _guarded(vocab, dim, vu.DT[dtype], pad, off)
        head.backward(hs, ws, tc, lse, gcu, grad_hidden=gh, grad_weight=gw)
        vu.check("grad_hidden", gh, want["gh"], want["gh_err"])
        vu.check("grad_weight", gw, want["gw"], want["gw_err"])
        ghu(), gwu()
        again = head.backward(hs, ws, tc, lse, gcu)
        assert torch.equal(again[0], gh) and torch.equal(again[1], gw), "two calls differ"
    # one gradient at a time, and added to what is there
    gw2 = base.cuda()
    none, gw2 = head.backward(hs, ws, tc, lse, gcu, grad_weight=gw2, accumulate=True, need=("weight",))
    both = vu.head(hc, w, t, scale, dtype, gc, base)
    assert none is None
    vu.check("accumulated grad_weight", gw2, both["gw"], both["gw_err"])
    gh2, none = head.backward(hs, ws, tc, lse, gcu, need=("hidden",))
    assert none is None and torch.equal(gh2, gh)
    head.close()


# shapes that fill the chip with large tiles: in the first product (words x
# rows), in grad_hidden (width x rows) and in grad_weight (width x words); the
# third has more rows than a piece of the vocabulary allows whole (several
# pieces, the last of odd size)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", [(2300, 6100, 136), (6200, 333, 2048), (300, 6301, 2048), (40_000, 4000, 64)])
def test_head_large(gr, dtype, n, vocab, dim):
    """The 64-bit formulas run on the GPU here (torch's fp64 products)."""
    h, w, t, g, (hc, gc) = (x if isinstance(x, tuple) else x.cuda() for x in _head_inputs(n, vocab, dim, dtype, 3 * n))
    want = vu.head(hc.cuda(), w, t, 1.0, dtype, gc.cuda())
    want = {k: v.cpu() for k, v in want.items()}
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)
    loss, lse = head.loss(h, w, t)
    vu.check("loss", loss, want["loss"], want["loss_err"])
    vu.check("lse", lse, want["lse"], want["lse_err"])
    gh, gw = head.backward(h, w, t, lse, g)
    vu.check("grad_hidden", gh, want["gh"], want["gh_err"])
    vu.check("grad_weight", gw, want["gw"], want["gw_err"])
    again = head.backward(h, w, t, lse, g)
    assert torch.equal(again[0], gh) and torch.equal(again[1], gw), "two calls differ"
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_more_words_than_a_piece_holds(gr, dtype):
    """Over two million words for few rows: a row of a piece's gradient stays
    within the offsets of a tile, so the vocabulary takes several pieces."""
    n, vocab, dim = 70, 2_200_003, 16
    h, w, t, g, (hc, gc) = (x if isinstance(x, tuple) else x.cuda() for x in _head_inputs(n, vocab, dim, dtype, 31))
    want = vu.head(hc.cuda(), w, t, 1.0, dtype, gc.cuda())
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)
    loss, lse = head.loss(h, w, t)
    gh, gw = head.backward(h, w, t, lse, g)
    for name, got in (("loss", loss), ("gh", gh), ("gw", gw)):
        vu.check(name, got, want[name].cpu(), want[name + "_err"].cpu())
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 40, 100])
def test_head_rows_and_words_of_far_sizes(gr, dtype, n):
    """Rows and words many powers of two apart, and of zeros: each fp32 row is
    scaled by itself."""
    vocab, dim = 700, 160
    h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, dtype, 55 + n)
    size = 2.0 ** torch.randint(-30, 31, (n, 1), generator=_gen(1))
    back = 2.0 ** torch.randint(-12, 4, (vocab, 1), generator=_gen(2))
    h, hc = (h.float() * size).to(h.dtype), (hc.float() * size).to(h.dtype)
    w = (w.float() * back / size.max()).to(w.dtype)
    hc[n // 2] = 0
    h[n // 2] = 0
    w[5] = 0
    want = vu.head(hc, w, t, 64.0, dtype, gc)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype, scale=64.0)
    loss, lse = head.loss(h.cuda(), w.cuda(), t.cuda())
    vu.check("loss", loss, want["loss"], want["loss_err"])
    gh, gw = head.backward(h.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
    vu.check("grad_hidden", gh, want["gh"], want["gh_err"])
    vu.check("grad_weight", gw, want["gw"], want["gw_err"])
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_fewer_rows_than_planned(gr, dtype):
    """One handle, calls of every size up to its most: each as a handle of its own."""
    vocab, dim = 400, 128
    head = gr.Head(vocab, dim, max_rows=600, dtype=dtype)
    for n in (600, 1, 0, 16, 129, 5, 333):
        h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, dtype, n + 1)
        want = vu.head(hc, w, t, 1.0, dtype, gc) if n else None
        loss, lse = head.loss(h.cuda(), w.cuda(), t.cuda())
        gh, gw = head.backward(h.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
        if n == 0:
            assert loss.numel() == 0 and bool((gw == 0).all())
            continue
        vu.check("loss", loss, want["loss"], want["loss_err"])
        vu.check("grad_hidden", gh, want["gh"], want["gh_err"])
        vu.check("grad_weight", gw, want["gw"], want["gw_err"])
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 200])
def test_head_no_row_has_a_target(gr, dtype, n):
    vocab, dim = 150, 96
    h = torch.full((n, dim), float("nan"), dtype=vu.DT[dtype], device="cuda")
    w = torch.randn(vocab, dim, generator=_gen(4)).to(vu.DT[dtype]).cuda()
    t = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)
    loss, lse = head.loss(h, w, t)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    base = torch.randn(vocab, dim, generator=_gen(5)).to(vu.DT[dtype]).cuda()
    gw = base.clone()
    gh, _ = head.backward(h, w, t, lse, torch.full((n,), float("nan"), device="cuda"), grad_weight=gw, accumulate=True)
    assert bool((gh == 0).all()) and torch.equal(gw, base)
    gh, gw = head.backward(h, w, t, lse, torch.full((n,), float("nan"), device="cuda"))
    assert bool((gh == 0).all()) and bool((gw == 0).all())
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_far_logits(gr, dtype):
    """Logits of hundreds and rows whose target is all but certain or all but
    impossible: the maximum is taken out before the exponentials."""
    n, vocab, dim = 40, 333, 64
    h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, dtype, 77)
    h, hc = h * 60, hc * 60
    want = vu.head(hc, w, t, 4.0, dtype, gc)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype, scale=4.0)
    loss, lse = head.loss(h.cuda(), w.cuda(), t.cuda())
    vu.check("loss", loss, want["loss"], want["loss_err"])
    gh, gw = head.backward(h.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
    vu.check("grad_hidden", gh, want["gh"], want["gh_err"])
    vu.check("grad_weight", gw, want["gw"], want["gw_err"])
    head.close()


def test_head_gradient_against_differences(gr):
    """Central differences of the 64-bit loss along random directions."""
    n, vocab, dim = 37, 210, 48
    h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, "f32", 12)
    head = gr.Head(vocab, dim, max_rows=n)
    _, lse = head.loss(h.cuda(), w.cuda(), t.cuda())
    gh, gw = (x.double().cpu() for x in head.backward(h.cuda(), w.cuda(), t.cuda(), lse, g.cuda()))
    ok = (t >= 0) & (t < vocab)

    def total(hh, ww):
        return float((vu.head(hh, ww, t, 1.0, "f32")["loss"] * torch.where(ok, gc.double(), 0.0)).sum())

    gen, eps = _gen(5), 1e-5
    for _ in range(6):
        dh = torch.randn(n, dim, generator=gen, dtype=torch.float64)
        dw = torch.randn(vocab, dim, generator=gen, dtype=torch.float64)
        num = (total(hc.double() + eps * dh, w.double() + eps * dw) - total(hc.double() - eps * dh, w.double() - eps * dw)) / (2 * eps)
        ana = float((gh * dh).sum() + (gw * dw).sum())
        # fp32 gradients of relative error about 1e-6 of their norms, and the
        # difference's eps^2 term (third derivatives of order the direction's norm cubed: below 1e-6)
        scale = float((gh.norm() * dh.norm()) + (gw.norm() * dw.norm()))
        assert abs(num - ana) <= 1e-5 * scale, (num, ana)
    head.close()


# ---------------------------------------------------------- used together

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_search_path_gradient_to_a_tied_table(gr, dtype):
    """A search whose logits come from a table, its surrogate backward, the
    head's backward over the paths and the lookup's backward into one gradient
    of the tied table, against the same chain in 64 bits."""
    B, K, V, D, T = 2, 6, 90, 64, 3
    gen = _gen(21)
    w = (torch.randn(V, D, generator=gen) * 0.3).to(vu.DT[dtype])
    wc = w.cuda()
    n = B * K
    emb = gr.Embedding(V, D, max_tokens=n, dtype=dtype, scale=8.0)
    head = gr.Head(V, D, max_rows=n, dtype=dtype)
    beam = gr.Beam(B, K, V, T, dtype="f32")
    tokens = torch.zeros(B, K, dtype=torch.int32, device="cuda")  # a start word
    fed, states = [], []
    for _ in range(T):
        x = emb.lookup(tokens, wc)  # the "model": each beam's state is its last word's row
        fed.append(tokens)
        states.append(x)
        beam.step((x.float().reshape(n, D) @ wc.float().T).reshape(B, K, V).contiguous())
        tokens = beam.state()["tokens"][beam.step_index - 1].contiguous()
    paths = beam.backward(torch.rand(B, K, generator=gen).cuda())
    gw = torch.zeros(V, D, dtype=vu.DT[dtype], device="cuda")
    want, err = torch.zeros(V, D, dtype=torch.float64), torch.zeros(V, D, dtype=torch.float64)
    for t in range(T):
        slot, word = paths["path_slot"][t], paths["path_token"][t].contiguous()
        rows = slot.clamp(min=0).long()[..., None].expand(-1, -1, D)
        h = states[t].gather(1, rows).contiguous()
        src = fed[t].gather(1, slot.clamp(min=0).long()).contiguous()
        loss, lse = head.loss(h, wc, word)
        up = (-paths["weight"]).contiguous()
        gh, _ = head.backward(h, wc, word, lse, up, grad_weight=gw, accumulate=True)
        emb.backward(src, gh, grad_weight=gw, accumulate=True)
        r = vu.head(h.cpu().reshape(n, D), w, word.cpu(), 1.0, dtype, up.cpu())
        vu.check("loss", loss, r["loss"], r["loss_err"])
        s, es = vu.scatter(src.cpu(), gh.cpu(), V, 8.0, dtype)
        want, err = want + r["gw"] + s, err + r["gw_err"] + es + 2 * vu.UT[dtype] * (want.abs() + r["gw"].abs() + s.abs())
    vu.check("tied gradient", gw, want, err)
    # each final beam's score is the sum of its steps' log-probabilities (step t's loss is -log p)
    assert bool(torch.isfinite(beam.state()["scores"]).all())
    for x in (emb, head, beam):
        x.close()


def test_loss_is_the_beam_steps_normaliser(gr):
    """The head's lse of fp32 rows is the step's lse of their logits, within the
    roundings of the two."""
    B, K, V, D = 2, 5, 1280, 64
    gen = _gen(8)
    h, w = torch.randn(B * K, D, generator=gen), torch.randn(V, D, generator=gen) * 0.2
    beam = gr.Beam(B, K, V, 2)
    logits = (h.double() @ w.double().T).float().reshape(B, K, V).cuda()
    beam.step(logits)
    beam.step(logits)  # every slot is live at the second step
    head = gr.Head(V, D, max_rows=B * K)
    _, lse = head.loss(h.cuda(), w.cuda(), torch.zeros(B * K, dtype=torch.int32, device="cuda"))
    r = vu.head(h, w, torch.zeros(B * K), 1.0, "f32")
    vu.check("lse", lse, r["lse"], r["lse_err"])
    vu.check("lse of the step", beam.state()["lse"].flatten(), r["lse"], r["lse_err"])
    head.close(), beam.close()


# ------------------------------------------------- streams, graphs, refusals

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_on_a_side_stream_and_replayed_from_a_graph(gr, dtype):
    n, vocab, dim = 150, 300, 128
    h, w, t, g, _ = _head_inputs(n, vocab, dim, dtype, 5)
    h, w, t, g = h.cuda(), w.cuda(), t.cuda(), g.cuda()
    up = torch.randn(n, dim, generator=_gen(6)).to(vu.DT[dtype]).cuda()
    emb = gr.Embedding(vocab, dim, max_tokens=n, dtype=dtype)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)

    def step(stream=None):
        loss, lse = head.loss(h, w, t, stream=stream)
        gh, gw = head.backward(h, w, t, lse, g, stream=stream)
        x = emb.lookup(t, w, stream=stream)
        emb.backward(t, up, grad_weight=gw, accumulate=True, stream=stream)
        return loss, lse, gh, gw, x

    eager = [o.clone() for o in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = step(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, outs):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        for o in outs:
            o.fill_(3.0)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b), f"replay {i}"
        # new inputs in the same places: what a replay reads is the buffers
        h.mul_(1.0)
        torch.cuda.synchronize()
        for a, b in zip(eager, step()):
            assert torch.equal(a, b), f"eager call after replay {i}"
    emb.close(), head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(150, 300), (700, 900)])
def test_replay_reads_what_the_buffers_hold(gr, dtype, n, vocab):
    """A captured step replayed on other inputs, with another number of rows that
    have a target (none and all among them), is the eager step on those."""
    dim = 128
    emb = gr.Embedding(vocab, dim, max_tokens=n, dtype=dtype)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)
    h, w, t, g = (torch.zeros(s, dtype=d, device="cuda") for s, d in
                  (((n, dim), vu.DT[dtype]), ((vocab, dim), vu.DT[dtype]), ((n,), torch.int32), ((n,), torch.float32)))

    def step():
        loss, lse = head.loss(h, w, t)
        gh, gw = head.backward(h, w, t, lse, g)
        return loss, lse, gh, gw, emb.lookup(t, w), emb.backward(t, gh)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, absent in enumerate((0.2, 1.0, 0.0, 0.6)):
        hh, ww, tt, gg, _ = _head_inputs(n, vocab, dim, dtype, 40 + i, absent)
        for dst, src in ((h, hh), (w, ww), (t, tt), (g, gg)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for k, (a, b) in enumerate(zip(got, step())):
            assert torch.equal(a, b), f"replay {i}, output {k}"
    emb.close(), head.close()


def test_two_handles_on_two_streams(gr):
    """Handles do not share workspaces: work of two of them may overlap."""
    n, vocab, dim = 900, 3000, 256
    data = [_head_inputs(n, vocab, dim, "bf16", s) for s in (1, 2)]
    data = [tuple(x.cuda() for x in d[:4]) for d in data]
    heads = [gr.Head(vocab, dim, max_rows=n, dtype="bf16") for _ in data]
    embs = [gr.Embedding(vocab, dim, max_tokens=n, dtype="bf16") for _ in data]

    def step(i, stream=None):
        h, w, t, g = data[i]
        loss, lse = heads[i].loss(h, w, t, stream=stream)
        gh, gw = heads[i].backward(h, w, t, lse, g, stream=stream)
        return loss, gh, gw, embs[i].backward(t, gh, stream=stream)

    alone = [step(i) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(3):
        both = [step(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    for x in (*heads, *embs):
        x.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [65_546, 70_000])
def test_head_more_rows_than_a_pass(gr, dtype, n):
    """More rows than one pass of the loss takes: the last pass is of few rows or
    of many."""
    vocab, dim = 200, 24
    h, w, t, g, (hc, gc) = (x if isinstance(x, tuple) else x.cuda() for x in _head_inputs(n, vocab, dim, dtype, 6))
    want = vu.head(hc.cuda(), w, t, 1.0, dtype, gc.cuda())
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype)
    loss, lse = head.loss(h, w, t)
    gh, gw = head.backward(h, w, t, lse, g)
    for name, got in (("loss", loss), ("lse", lse), ("gh", gh), ("gw", gw)):
        vu.check(name, got, want[name].cpu(), want[name + "_err"].cpu())
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim,scale", [(70, 90, 20_000, 1.0), (5, 40, 20_000, 1.0), (100, 300, 64, -0.75),
                                               (20, 300, 64, -0.75), (100, 300, 64, 1e-20), (3, 300, 64, 1e-20)])
def test_head_wide_rows_and_odd_scales(gr, dtype, n, vocab, dim, scale):
    scale = float(np.float32(scale))
    h, w, t, g, (hc, gc) = _head_inputs(n, vocab, dim, dtype, 3)
    want = vu.head(hc, w, t, scale, dtype, gc)
    head = gr.Head(vocab, dim, max_rows=n, dtype=dtype, scale=scale)
    loss, lse = head.loss(h.cuda(), w.cuda(), t.cuda())
    gh, gw = head.backward(h.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
    for name, got in (("loss", loss), ("lse", lse), ("gh", gh), ("gw", gw)):
        vu.check(name, got, want[name], want[name + "_err"])
    head.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [7, 100, 1500])
def test_scoring_head_is_the_training_heads_loss(gr, dtype, n):
    h, w, t, g, _ = _head_inputs(n, 1000, 100, dtype, 8)
    h, w, t = h.cuda(), w.cuda(), t.cuda()
    full, score = (gr.Head(1000, 100, max_rows=n, dtype=dtype, backward=b) for b in (True, False))
    for a, b in zip(full.loss(h, w, t), score.loss(h, w, t)):
        assert torch.equal(a, b)
    full.close(), score.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", [(1_200_000, 70_000, 8), (3000, 5_000_000, 4), (20_000, 5000, 1024), (513, 2047, 8),
                                         (600, 2048, 8), (900, 3, 6000), (1025, 70_000, 150), (2048, 1, 40),
                                         (2048, 333, 25), (2049, 333, 25)])
def test_embedding_of_many(gr, dtype, n, vocab, dim):
    """Sorts by one workgroup and of one, two and three passes, tiles of more than a few rows, whole
    rows to a thread group, and lookups of four rows a group."""
    gen = _gen(n)
    t = _tokens(n, vocab, gen, 0.1)
    ok = (t >= 0) & (t < vocab)
    w = torch.randn(vocab, dim, generator=gen).to(vu.DT[dtype])
    g = torch.randn(n, dim, generator=gen).to(vu.DT[dtype])
    e = gr.Embedding(vocab, dim, max_tokens=n, dtype=dtype, scale=0.5)
    want = torch.where(ok[:, None], w[t.clamp(0, vocab - 1).long()].float() * 0.5, 0.0).to(vu.DT[dtype])
    assert torch.equal(e.lookup(t.cuda(), w.cuda()).cpu(), want)
    ref, err = vu.scatter(t, g, vocab, 0.5, dtype)
    vu.check("grad_weight", e.backward(t.cuda(), g.cuda()), ref, err)
    e.close()


def test_workspace_that_does_not_fit(gr):
    """An allocation that fails is an error of init; nothing of it stays behind."""
    free = torch.cuda.mem_get_info()[0]
    with pytest.raises(gr.GrError) as e:
        gr.Head(1 << 30, 64, max_rows=1 << 20, dtype="bf16")  # 8 TB of parts
    assert e.value.status == gr._lib.GR_ERR_OUT_OF_MEMORY
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] >= free - (64 << 20)
    head = gr.Head(48, 64, max_rows=4)
    x = torch.zeros(4, 64, device="cuda")
    loss, _ = head.loss(x, torch.zeros(48, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
    # log 48 within fp32 roundings of a sum of 48 ones and a logarithm
    assert abs(float(loss[0]) - float(np.log(48.0))) < 1e-5
    head.close()


def test_refusals(gr):
    E, H = gr.Embedding(40, 16, max_tokens=8), gr.Head(40, 16, max_rows=8, dtype="bf16")
    w = torch.zeros(40, 16, device="cuda")
    wb = w.bfloat16()
    t = torch.zeros(8, dtype=torch.int32, device="cuda")
    hb = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros(8, device="cuda")
    with pytest.raises(TypeError):
        E.lookup(t.long(), w)
    with pytest.raises(TypeError):
        E.lookup(t.cpu(), w)
    with pytest.raises(TypeError):
        E.lookup(t, wb)
    with pytest.raises(ValueError):
        E.lookup(t, w[:39])
    with pytest.raises(ValueError):
        E.lookup(t, w[:, :15])
    with pytest.raises(ValueError):
        E.lookup(t, w.t().contiguous().t())
    with pytest.raises(ValueError):
        E.lookup(t[::2], w)
    with pytest.raises(ValueError):
        E.lookup(t, w[:1].expand(40, 16))
    with pytest.raises(gr.GrError) as e:
        E.lookup(torch.zeros(9, dtype=torch.int32, device="cuda"), w)
    assert e.value.status == gr._lib.GR_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        E.backward(t, w[:8], accumulate=True)
    with pytest.raises(ValueError):
        E.backward(t, w[:7])
    with pytest.raises(ValueError):
        H.loss(hb[:7], wb, t)
    with pytest.raises(TypeError):
        H.loss(hb.float(), wb, t)
    with pytest.raises(ValueError):
        H.backward(hb, wb, t, f[:7], f)
    with pytest.raises(ValueError):
        H.backward(hb, wb, t, f, f, need=())
    with pytest.raises(ValueError):
        H.backward(hb, wb, t, f, f, need=("bias",))
    with pytest.raises(ValueError):
        H.backward(hb, wb, t, f, f, accumulate=True)
    big = torch.zeros(2, (1 << 22) + 1, dtype=torch.float32, device="cuda")
    one = gr.Embedding(2, 16, max_tokens=8)
    with pytest.raises(gr.GrError):
        one.lookup(t, big[:, :16])  # rows further apart than 2^22 elements
    S = gr.Head(40, 16, max_rows=8, dtype="bf16", backward=False)
    _, lse = S.loss(hb, wb, t)
    with pytest.raises(gr.GrError) as e:
        S.backward(hb, wb, t, lse, f)
    assert e.value.status == gr._lib.GR_ERR_UNSUPPORTED
    S.close()
    with pytest.raises(ValueError):
        S.loss(hb, wb, t)
    torch.cuda.synchronize()
