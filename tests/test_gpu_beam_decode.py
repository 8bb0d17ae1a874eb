"""Prompts in chunks, beams forked from them, and steps of attention, selection and reordering as one run over one pool.

A row of the pool depends on its token and position alone here (every layer's projections are looked up by token), so each beam's rows,
read through its table at the end, are bit for bit those of its whole sequence put into a fresh pool at once; its last output is
that sequence's within the calls' tolerances (two roundings to bf16, and the single-part weights of a chunk: 3 x 2^-8 of the
mean |v|), and the scores are the sums of the log-probabilities along it.
"""

import numpy as np
import pytest
import torch

from tests import paged_common as C

pytestmark = pytest.mark.gpu
LAYERS, HQ, HKV, D, VOCAB = 2, 8, 2, 64, 1000


class Model:
    def __init__(self, cuda, seed=0):
        g = torch.Generator().manual_seed(seed)
        make = lambda *s: torch.randn(*s, generator=g).bfloat16().to(cuda)      # noqa: E731
        self.q, self.k, self.v = (make(LAYERS, VOCAB, h, D) for h in (HQ, HKV, HKV))
        self.head = (torch.randn(LAYERS * HQ * D, VOCAB, generator=g) * 0.1).bfloat16().to(cuda)


def decoder(cuda, K, batch, max_rows, n_pages, **kw):
    from attention_kv_cache_gb300.pipeline import PagedDecoder
    return PagedDecoder(n_layers=LAYERS, h_q=HQ, h_kv=HKV, head_dim=D, batch=batch, max_rows=max_rows, n_pages=n_pages, page_size=16,
                        rope=K.RopeScaling(K.ROPE_PLAIN, 10000.0, 1.0, 1.0, 4.0, 256), device=cuda, **kw)


def chunk(dec, model, tokens, n_new):
    """tokens [max_tokens] of a step's requests one after another; the last layer's outputs of every layer."""
    dec.begin_chunk(n_new)
    return [dec.chunk_layer(x, model.q[x, tokens], model.k[x, tokens], model.v[x, tokens]).clone() for x in range(LAYERS)]


def step(dec, model, tokens):
    dec.begin()
    return torch.stack([dec.layer(x, model.q[x, tokens], model.k[x, tokens], model.v[x, tokens]).clone() for x in range(LAYERS)], 1)


@pytest.mark.parametrize("cache_dtype", [None, torch.float8_e4m3fn])
def test_beam_search(cuda, cache_dtype):
    from attention_kv_cache_gb300 import kvsel as K
    from attention_kv_cache_gb300.pipeline import BeamSelector
    sets, beams, steps, prompts = 3, 4, 21, [37, 64, 150]
    model, batch = Model(cuda), sets * beams
    scales = None if cache_dtype is None else tuple((0.02 + torch.zeros(LAYERS, HKV)).to(cuda) for _ in range(2))
    kw = dict(cache_dtype=cache_dtype, scales=scales)
    dec = decoder(cuda, K, batch, 200, 120, max_tokens=160, beams=beams, **kw)
    rng = np.random.default_rng(3)
    text = [rng.integers(0, VOCAB, n) for n in prompts]
    # the prompts into every set's first beam, all but their last token, in chunks of uneven shares
    done = [0] * sets
    for share in ([20, 30, 100], [16, 33, 49]):
        part = [t[a:a + n] for t, a, n in zip(text, done, share)]
        tokens = torch.zeros(160, dtype=torch.int64)
        flat = np.concatenate(part)
        tokens[:len(flat)] = torch.from_numpy(flat)
        n_new = torch.zeros(batch, dtype=torch.int64)
        n_new[::beams] = torch.tensor(share)
        chunk(dec, model, tokens.to(cuda), n_new.to(cuda))
        done = [a + n for a, n in zip(done, share)]
    assert done == [n - 1 for n in prompts]
    dec.fork()
    assert dec.lens.tolist() == [n - 1 for n in prompts for _ in range(beams)]
    pick = BeamSelector(sets=sets, beams=beams, n_out=beams, vocab=VOCAB, device=cuda)
    scores = torch.full((sets, beams), float("-inf"), device=cuda)
    scores[:, 0] = 0.0
    tokens = torch.tensor([t[-1] for t in text for _ in range(beams)], device=cuda)
    ids = [[list(t) for _ in range(beams)] for t in text]
    for i in range(steps):
        o = step(dec, model, tokens)
        logits = (o.reshape(batch, -1) @ model.head).contiguous()
        found = pick.select(logits, scores)
        scores, parents, new = (x.clone() for x in found)
        logp = torch.log_softmax(logits.double(), -1).view(sets, beams, VOCAB)
        if i == 0:
            assert (parents == 0).all()
        dec.reorder(parents)
        tokens = new.flatten().long()
        ids = [[ids[s][p] + [t] for p, t in zip(ps, ts)] for s, (ps, ts) in enumerate(zip(parents.tolist(), new.tolist()))]
        assert (scores[:, :-1] >= scores[:, 1:]).all() and torch.isfinite(logp).all()
    o = step(dec, model, tokens)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.OK
    # pages: named or free, none lost
    lens = dec.lens.tolist()
    named = {int(x) for r, n in zip(dec.tables, lens) for x in r[:-(-n // 16)]}
    free = dec.free_pages[int(dec.free_head):].tolist()
    assert len(set(free)) == len(free) and not named & set(free) and len(named) + len(free) == 120
    # every beam's whole sequence at once
    for s in range(sets):
        fresh = decoder(cuda, K, beams, 200, 60, max_tokens=beams * len(ids[s][0]), **kw)
        n = len(ids[s][0])
        assert lens[s * beams:(s + 1) * beams] == [n] * beams
        out = chunk(fresh, model, torch.tensor([t for r in ids[s] for t in r], device=cuda),
                    torch.full((beams,), n, dtype=torch.int64, device=cuda))
        torch.cuda.synchronize()
        for b in range(beams):
            for mine, theirs in ((dec.k_cache, fresh.k_cache), (dec.v_cache, fresh.v_cache)):
                a, e = (x.view(torch.uint8)[:, t[b if x is theirs else s * beams + b, :-(-n // 16)].long()]
                        for x, t in ((mine, dec.tables), (theirs, fresh.tables)))
                a, e = (x.permute(0, 1, 3, 2, 4).flatten(1, 2)[:, :n] for x in (a, e))
                assert torch.equal(a, e), (s, b)
            for x in range(LAYERS):
                a, e = o[s * beams + b, x].float(), out[x][(b + 1) * n - 1].float()
                assert (a - e).abs().max() <= 3 * 2.0 ** -8 * max(1.0, e.abs().max().item())


def test_steps_are_captured_and_shared_rows_change_nothing(cuda):
    """A step of beams replayed from a graph, and the same steps without sharing: the same tokens are chosen."""
    from attention_kv_cache_gb300 import kvsel as K
    from attention_kv_cache_gb300.pipeline import BeamSelector
    sets, beams, model = 2, 4, Model(cuda, 5)
    batch, chosen = sets * beams, []
    for mode in ("eager", "graph", "unshared"):
        dec = decoder(cuda, K, batch, 160, 100, max_tokens=100, beams=beams)
        tokens = torch.from_numpy(np.random.default_rng(9).integers(0, VOCAB, 100)).to(cuda)
        n_new = torch.zeros(batch, dtype=torch.int64, device=cuda)
        n_new[::beams] = 50
        chunk(dec, model, tokens, n_new)
        dec.fork()
        if mode == "unshared":
            dec.share(None, None)
        pick = BeamSelector(sets=sets, beams=beams, n_out=beams, vocab=VOCAB, device=cuda)
        scores = torch.full((sets, beams), float("-inf"), device=cuda)
        scores[:, 0] = 0.0
        now = torch.full((batch,), 7, dtype=torch.int64, device=cuda)
        log = []

        def one():
            o = step(dec, model, now)
            s, p, t = pick.select((o.reshape(batch, -1) @ model.head).contiguous(), scores)
            dec.reorder(p)
            scores.copy_(s)
            now.copy_(t.flatten())

        one()
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        for _ in range(12):
            graph.replay() if mode == "graph" else one()
            log.append((now.clone(), scores.clone()))
        torch.cuda.synchronize()
        assert K.kvsel_read_device_error(dec.ws) == K.OK
        chosen.append(log)
    for (t0, s0), (t1, s1), (t2, s2) in zip(*chosen):
        assert torch.equal(t0, t1) and torch.equal(s0, s1)
        # (outputs round differently without sharing: near ties may fall the other way, the best beam's score may not)
        assert (s0[:, 0] - s2[:, 0]).abs().max() < 0.5


def test_a_side_stream(cuda):
    """Prompt, fork and steps on a stream of their own, behind what the current one holds."""
    from attention_kv_cache_gb300 import kvsel as K
    model, side, outs = Model(cuda, 2), torch.cuda.Stream(), []
    for stream in (None, side):
        dec = decoder(cuda, K, 4, 100, 40, max_tokens=40, beams=2)
        tokens = torch.arange(40, device=cuda)
        n_new = torch.tensor([17, 0, 23, 0], device=cuda)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            dec.begin_chunk(n_new, stream=stream)
            for x in range(LAYERS):
                dec.chunk_layer(x, model.q[x, tokens], model.k[x, tokens], model.v[x, tokens], stream=stream)
        dec.fork(stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        outs.append(step(dec, model, torch.tensor([1, 2, 3, 4], device=cuda)))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_refusals(cuda):
    from attention_kv_cache_gb300 import kvsel as K
    from attention_kv_cache_gb300.pipeline import BeamSelector
    dec = decoder(cuda, K, 4, 100, 40, max_tokens=40, beams=2)
    plain = decoder(cuda, K, 4, 100, 40)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=cuda)       # noqa: E731
    bad = [lambda: decoder(cuda, K, 5, 100, 40, beams=2), lambda: plain.begin_chunk(torch.zeros(4, dtype=torch.int64, device=cuda)),
           lambda: plain.chunk_layer(0, zeros(40, HQ, D), zeros(40, HKV, D), zeros(40, HKV, D)),
           lambda: dec.begin_chunk(torch.zeros(3, dtype=torch.int64, device=cuda)),
           lambda: dec.begin_chunk(torch.zeros(4, dtype=torch.int32, device=cuda)),
           lambda: dec.begin_chunk(torch.zeros(4, dtype=torch.int64)),
           lambda: dec.chunk_layer(0, zeros(39, HQ, D), zeros(40, HKV, D), zeros(40, HKV, D)),
           lambda: dec.chunk_layer(0, zeros(40, HQ, D), zeros(40, HQ, D), zeros(40, HKV, D)),
           lambda: plain.reorder(torch.zeros(4, 1, dtype=torch.int32, device=cuda)), lambda: plain.fork(),
           lambda: dec.reorder(torch.zeros(2, 2, dtype=torch.int64, device=cuda)),
           lambda: dec.reorder(torch.zeros(4, 1, dtype=torch.int32, device=cuda)),
           lambda: dec.reorder(torch.zeros(2, 4, dtype=torch.int32, device=cuda)[:, ::2]),
           lambda: dec.share(torch.zeros(3, dtype=torch.int64, device=cuda), torch.zeros(3, dtype=torch.int64, device=cuda)),
           lambda: dec.share(torch.zeros(3, dtype=torch.int32, device=cuda), torch.zeros(2, dtype=torch.int64, device=cuda))]
    pick = BeamSelector(sets=2, beams=2, n_out=4, vocab=50, device=cuda)
    scores = torch.zeros(2, 2, device=cuda)
    bad += [lambda: pick.select(zeros(4, 51), scores), lambda: pick.select(zeros(4, 50).float(), scores),
            lambda: pick.select(zeros(4, 64)[:, :50], scores), lambda: pick.select(zeros(4, 50), scores.double()),
            lambda: pick.select(zeros(4, 50), torch.zeros(4, device=cuda)),
            lambda: pick.select(zeros(4, 50), scores, torch.zeros(2, 2, device=cuda))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(i)
    with pytest.raises(K.KvselError):
        BeamSelector(sets=2, beams=2, n_out=65, vocab=50, device=cuda)


def test_refusals_of_other_layouts_and_devices(cuda):
    """Views that are not dense, whose neighbours the kernels would read, and tensors on the host."""
    from attention_kv_cache_gb300 import kvsel as K
    from attention_kv_cache_gb300.pipeline import BeamSelector
    dec = decoder(cuda, K, 4, 100, 40, max_tokens=40, beams=2)
    long = torch.zeros(8, dtype=torch.int64, device=cuda)
    pick = BeamSelector(sets=2, beams=2, n_out=4, vocab=50, device=cuda)
    logits, scores = torch.zeros(4, 50, dtype=torch.bfloat16, device=cuda), torch.zeros(2, 2, device=cuda)
    ended = torch.zeros(2, 2, dtype=torch.uint8, device=cuda)
    for f in (lambda: dec.begin_chunk(long[::2]), lambda: dec.share(long[:6:2], long[:2]), lambda: dec.share(long[:3], long[:4:2]),
              lambda: pick.select(logits.cpu(), scores), lambda: pick.select(logits, scores.cpu()),
              lambda: pick.select(logits, scores, ended.cpu()), lambda: pick.select(logits, scores.t(), ended[:, :1].expand(2, 2))):
        with pytest.raises(ValueError):
            f()
    pick.select(logits, scores, ended)
    torch.cuda.synchronize()


def graph_of(run):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
    torch.cuda.current_stream().wait_stream(side)
    return g


def test_captured_step_reads_the_next_fork(cuda):
    """A step captured behind one prompt's fork runs behind another's: shorter, so that the first one's shared rows are too many."""
    from attention_kv_cache_gb300 import kvsel as K
    model, beams = Model(cuda), 3
    make = lambda: decoder(cuda, K, beams, 128, 40, max_tokens=100, beams=beams)     # noqa: E731
    dec, tokens = make(), torch.tensor([5, 6, 7], device=cuda)
    out = torch.empty((beams, LAYERS, HQ, D), dtype=torch.bfloat16, device=cuda)
    text = torch.randint(0, VOCAB, (100,), generator=torch.Generator().manual_seed(2)).to(cuda)

    def begin(d, n):
        d.lens.zero_()
        d.free_pages.copy_(torch.arange(40, dtype=torch.int32, device=cuda))
        d.free_head.zero_()
        chunk(d, model, text, torch.tensor([n, 0, 0], device=cuda))
        d.fork()

    begin(dec, 100)
    before = dec.ws.data_ptr()
    g = graph_of(lambda: out.copy_(step(dec, model, tokens)))
    begin(dec, 41)
    assert dec.ws.data_ptr() == before
    g.replay()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.OK and dec.lens.tolist() == [42] * beams
    other = make()
    begin(other, 41)
    assert torch.equal(out, step(other, model, tokens))


def test_an_outgrown_workspace_stays(cuda):
    """Sharing may need more room: the room that captured steps use is not given to anyone else."""
    from attention_kv_cache_gb300 import kvsel as K
    model, batch = Model(cuda), 4
    dec, tokens = decoder(cuda, K, batch, 64, 16), torch.tensor([1, 2, 3, 4], device=cuda)
    for _ in range(20):
        o = step(dec, model, tokens)
    lens = dec.lens.clone()
    start, n = dec.ws.data_ptr(), dec.ws.numel()
    out = torch.empty_like(o)
    g = graph_of(lambda: out.copy_(step(dec, model, tokens)))
    dec.share(torch.arange(batch + 1, device=cuda), torch.full((batch,), 16, device=cuda))
    assert dec.ws.numel() > n
    others = [torch.full((n + K.WS_ALIGN,), 255, dtype=torch.uint8, device=cuda) for _ in range(8)]
    assert all(x.data_ptr() + x.numel() <= start or x.data_ptr() >= start + n for x in others)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dec.lens, lens + 1) and all((x == 255).all() for x in others)
    fresh = decoder(cuda, K, batch, 64, 16)
    for _ in range(21):
        want = step(fresh, model, tokens)
    assert torch.equal(out, want)
