"""Selection, compaction and then decode steps over the paged pool, as one run: the operators after one another.

Each step's rows in the pool and its queries are held to the definition (norm, rotation, one rounding), and its
attention to the fp64 softmax over the rows the pool then holds; tolerances are those of the single calls.
"""

import numpy as np
import pytest
import torch

from attention_kv_cache_gb300 import synth as S
from oracle import paged_oracle as O
from tests import paged_common as C
from tests.test_gpu_paged_append import near

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _setup(cuda, cache_dtype=None, steps=20):
    from attention_kv_cache_gb300 import kvsel as K
    from attention_kv_cache_gb300.pipeline import PagedDecoder, Pipeline, pack
    w = S.scaled(S.TINY, n_layers=2, prefix_lens=[300, 411, 290])
    inp = S.make_inputs(w, "cpu")
    q, k, v = pack(inp, cuda)
    pipe = Pipeline(w, cuda)
    pipe.run(q, k, v)
    rows, g = pipe.k_out.shape[3], torch.Generator().manual_seed(8)
    P = 16
    norms = [tuple((1 + 0.1 * torch.randn(w.head_dim, generator=g)).bfloat16().to(cuda) for _ in range(2))
             for _ in range(w.n_layers)]
    scales = None
    if cache_dtype is not None:
        scales = tuple((0.02 + 0.02 * torch.rand(w.n_layers, w.h_kv, generator=g)).to(cuda) for _ in range(2))
    dec = PagedDecoder(n_layers=w.n_layers, h_q=w.h_q, h_kv=w.h_kv, head_dim=w.head_dim, batch=w.batch,
                       max_rows=rows + steps, n_pages=w.batch * -(-(rows + steps) // P) + 2, page_size=P,
                       cache_dtype=cache_dtype, rope=K.RopeScaling(K.ROPE_BANDED, 10000.0, 4.0, 1.0, 4.0, 256),
                       norms=norms, scales=scales, device=cuda)
    text = [L + w.window for L in w.prefix_lens]
    dec.admit(pipe.k_out, pipe.v_out, text)
    xs = [torch.randn(w.n_layers, w.batch, w.h_q + 2 * w.h_kv, w.head_dim, generator=g).bfloat16().to(cuda)
          for _ in range(steps)]
    return K, w, pipe, dec, text, rows, xs


def _pool_rows(dec, pool, layer, b, n):
    t = torch.arange(n, device=pool.device)
    page = dec.tables[b].long()[t // dec.P]
    x = pool[layer].view(torch.uint8) if pool.element_size() == 1 else pool[layer]
    return C.f64(x[page, :, t % dec.P].contiguous().view(pool.dtype))          # [n, h_kv, d]


@pytest.mark.parametrize("cache_dtype", [None, torch.float8_e4m3fn])
def test_decode_goes_on_from_a_selection(cuda, cache_dtype):
    K, w, pipe, dec, text, rows, xs = _setup(cuda, cache_dtype)
    kind = "bf16" if cache_dtype is None else "e4m3"
    freq, factor = O.rope_freqs(w.head_dim, "banded", 10000.0, 4.0, 1.0, 4.0, 256)
    G = w.h_q // w.h_kv
    # the admitted rows: the compacted caches' own (in 16 bits exactly)
    for layer in range(w.n_layers):
        for pool, src, sc in ((dec.k_cache, pipe.k_out, 0), (dec.v_cache, pipe.v_out, 1)):
            for b in range(w.batch):
                got, want = _pool_rows(dec, pool, layer, b, rows), C.f64(src[b, layer]).transpose(1, 0, 2)
                if dec.scales is None:
                    assert np.array_equal(got, want)
                else:
                    want = want / C.f64(dec.scales[sc][layer])[:, None]
                    near(got, want, np.abs(want), kind, "admitted")
    for step, x in enumerate(xs):
        dec.begin()
        n = rows + step + 1
        assert dec.lens.tolist() == [n] * w.batch
        pos = np.array([t + step for t in text])
        assert dec.positions.tolist() == pos.tolist()
        for layer in range(w.n_layers):
            q, k, v = x[layer][:, :w.h_q], x[layer][:, w.h_q:w.h_q + w.h_kv], x[layer][:, w.h_q + w.h_kv:]
            o = C.f64(dec.layer(layer, q, k, v))
            if step % 7 and step < len(xs) - 1:
                continue
            qw, kw = dec.norms[layer]
            f32 = float(np.float32(factor))
            qr, size = O.norm_rope(C.f64(q), pos, freq, f32, "half", C.f64(qw), 0.0, 1e-6)
            near(C.f64(dec.q_out), qr, size, "bf16", "q")
            kr, ksize = O.norm_rope(C.f64(k), pos, freq, f32, "half", C.f64(kw), 0.0, 1e-6)
            vr = C.f64(v)
            sk, sv = ((1.0, 1.0) if dec.scales is None else (C.f64(s[layer])[:, None] for s in dec.scales))
            for b in range(w.batch):
                kp, vp = (_pool_rows(dec, p, layer, b, n) for p in (dec.k_cache, dec.v_cache))
                near(kp[-1], (kr / sk)[b], (ksize / sk)[b], kind, "k")
                near(vp[-1], (vr / sv)[b], np.abs(vr / sv)[b], kind, "v")
                kp, vp = kp * sk, vp * sv
                for h in range(w.h_kv):
                    hs = slice(h * G, (h + 1) * G)
                    qh = C.f64(dec.q_out)[b, hs]
                    want, _, mass, zmax = O.paged_attend(qh, kp[:, h], vp[:, h], w.head_dim ** -0.5)
                    dz = 2 * U * (w.head_dim + 8) * zmax
                    dz += U * w.head_dim ** 0.5 * np.abs(qh).max() * np.abs(kp).max()
                    tol = 2.0 ** -8 * np.abs(want) + 2 * (dz + 2.0 ** -17 + 2 * U * (n + 64)) * mass + 2 * U * n * np.abs(vp).max()
                    assert (np.abs(o[b, hs] - want) <= tol).all(), (step, layer, b, h)
    assert K.kvsel_read_device_error(dec.ws) == K.OK
    pages = dec.tables[:, :-(-(rows + len(xs)) // dec.P)].reshape(-1).tolist()
    assert len(set(pages)) == len(pages)                                      # no page serves two requests


def test_a_captured_step_replays_to_the_eager_bits(cuda):
    K, w, _, eager, _, _, xs = _setup(cuda, steps=9)
    *_, dec, _, _, _ = _setup(cuda, steps=9)
    x = torch.empty_like(xs[0])
    outs = torch.empty((w.n_layers, w.batch, w.h_q, w.head_dim), dtype=torch.bfloat16, device=cuda)

    def step(d, dst):
        d.begin()
        for layer in range(w.n_layers):
            y = x[layer]
            dst[layer].copy_(d.layer(layer, y[:, :w.h_q], y[:, w.h_q:w.h_q + w.h_kv], y[:, w.h_q + w.h_kv:]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(dec, outs)
    for i in range(9):
        x.copy_(xs[i])
        g.replay()
        want = torch.empty_like(outs)
        step(eager, want)
        torch.cuda.synchronize()
        assert torch.equal(outs, want), i
        assert torch.equal(dec.lens, eager.lens) and torch.equal(dec.tables, eager.tables)
    assert K.kvsel_read_device_error(dec.ws) == K.OK and K.kvsel_read_device_error(eager.ws) == K.OK


def test_a_pool_that_runs_out_stops_the_step(cuda):
    """No page left: the step assigns nothing, its rows are padding, and the pool keeps its bits."""
    K, w, _, dec, _, rows, xs = _setup(cuda, steps=40)
    dec.free_pages = dec.free_pages[:int(dec.free_head)].clone()
    held = -(-rows // dec.P) * dec.P
    for _ in range(held - rows):                       # the last pages fill up
        dec.begin()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.OK
    before = dec.k_cache.clone()
    dec.begin()
    x = xs[0][0]
    dec.layer(0, x[:, :w.h_q], x[:, w.h_q:w.h_q + w.h_kv], x[:, w.h_q + w.h_kv:])
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.ERR_INVALID_ARG
    assert dec.lens.tolist() == [held] * w.batch and dec.slots.tolist() == [-1] * w.batch
    assert torch.equal(dec.k_cache.view(torch.int16), before.view(torch.int16))
