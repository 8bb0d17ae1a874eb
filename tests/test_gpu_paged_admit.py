"""PagedDecoder.admit on any stream: the rows, lengths and positions are right whatever the streams are busy with."""

import contextlib

import pytest
import torch

from tests import paged_common as C

pytestmark = pytest.mark.gpu
BUSY = 40_000_000           # clocks, about 20 ms


def _decoder(cuda, batch=3, rows=37, n_layers=2, h_kv=2, d=64, P=16, seed=0, **kw):
    from attention_kv_cache_gb300.pipeline import PagedDecoder
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(batch, n_layers, h_kv, rows, d, generator=g).bfloat16().to(cuda) for _ in range(2))
    dec = PagedDecoder(n_layers=n_layers, h_q=2 * h_kv, h_kv=h_kv, head_dim=d, batch=batch, max_rows=rows + 40,
                       n_pages=batch * -(-(rows + 40) // P) + 1, page_size=P, device=cuda, **kw)
    return dec, k, v


def _rows(dec, pool, layer, b, n):
    t = torch.arange(n, device=pool.device)
    return pool[layer][dec.tables[b].long()[t // dec.P], :, t % dec.P].transpose(0, 1)      # [h_kv, n, d]


def _check(dec, k, v, text):
    from attention_kv_cache_gb300 import kvsel as K
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.OK
    n = k.shape[3]
    assert dec.lens.tolist() == [n] * dec.batch
    assert (dec.lens + dec.pos_offset).tolist() == text
    for layer in range(dec.n_layers):
        for b in range(dec.batch):
            assert torch.equal(_rows(dec, dec.k_cache, layer, b, n), k[b, layer])
            assert torch.equal(_rows(dec, dec.v_cache, layer, b, n), v[b, layer])
    dec.begin()
    torch.cuda.synchronize()
    assert dec.positions.tolist() == text and K.kvsel_read_device_error(dec.ws) == K.OK


@pytest.mark.parametrize("given", ["stream", "handle", "current"])
@pytest.mark.parametrize("busy", ["main", "side", "neither"])
@pytest.mark.parametrize("device_text", [False, True])
def test_another_stream(cuda, given, busy, device_text):
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for seed in range(3):
        text = [90 + seed, 55, 37]
        if busy == "main":
            torch.cuda._sleep(BUSY)
        dec, k, v = _decoder(cuda, seed=seed)                # its buffers' first values are the main stream's
        texts = torch.tensor(text).to(cuda) if device_text else text
        if busy == "side":
            side.wait_stream(main)
            with torch.cuda.stream(side):
                torch.cuda._sleep(BUSY)
        with torch.cuda.stream(side) if given == "current" else contextlib.nullcontext():
            if given == "current":
                side.wait_stream(main)
            dec.admit(k, v, texts, stream={"stream": side, "handle": side.cuda_stream, "current": None}[given])
        # memory that admit gave back must not be handed out under its kernels
        spoil = [torch.full((n,), 2 ** 62, dtype=torch.int64, device=cuda) for n in (dec.batch, dec.batch * k.shape[3]) * 20]
        _check(dec, k, v, text)
        del spoil


def test_a_captured_admission(cuda):
    """Admission within a capture, on the capturing stream."""
    dec, k, v = _decoder(cuda)
    texts = torch.tensor([90, 55, 37], device=cuda)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.admit(k, v, texts)
    assert dec.lens.tolist() == [0, 0, 0]
    g.replay()
    _check(dec, k, v, texts.tolist())


@pytest.mark.parametrize("first", [1, 16, 20])
def test_a_second_admission_goes_on_behind_the_first(cuda, first):
    """Rows in two parts are rows at once, and the next row's position is that of the whole text."""
    dec, k, v = _decoder(cuda)
    dec.admit(k, v, [40, 41, 42], rows=first)
    torch.cuda.synchronize()
    assert (dec.lens + dec.pos_offset).tolist() == [40, 41, 42]
    dec.admit(k[:, :, :, first:], v[:, :, :, first:], [90, 55, 37])
    _check(dec, k, v, [90, 55, 37])


def test_admission_behind_decoded_rows(cuda):
    dec, k, v = _decoder(cuda)
    dec.admit(k, v, [90, 55, 37], rows=10)
    for _ in range(5):
        dec.begin()
    dec.admit(k[:, :, :, 10:20], v[:, :, :, 10:20], [200, 201, 202])
    torch.cuda.synchronize()
    assert dec.lens.tolist() == [25] * 3 and (dec.lens + dec.pos_offset).tolist() == [200, 201, 202]
    for b in range(3):
        assert torch.equal(_rows(dec, dec.k_cache, 1, b, 25)[:, 15:], k[b, 1, :, 10:20])


def test_an_admission_of_no_rows(cuda):
    dec, k, v = _decoder(cuda)
    dec.admit(k, v, [5, 6, 7], rows=0)
    dec.begin()
    torch.cuda.synchronize()
    assert dec.lens.tolist() == [1, 1, 1] and dec.positions.tolist() == [5, 6, 7]


def test_whole_texts_under_a_window(cuda):
    dec, k, v = _decoder(cuda, window=20, slopes=torch.ones(4, device=cuda))
    with pytest.raises(ValueError):
        dec.admit(k, v, [38, 37, 37])
    side = torch.cuda.Stream()
    torch.cuda._sleep(BUSY)
    dec.admit(k, v, [37, 37, 37], stream=side)
    torch.cuda.synchronize()
    dec.begin()
    dec.admit(k, v, torch.tensor([45, 45, 45], device=cuda), rows=7)
    with pytest.raises(ValueError):
        dec.admit(k, v, [45, 45, 45], rows=1)
    torch.cuda.synchronize()
    assert dec.lens.tolist() == [45, 45, 45] and dec.pos_offset.tolist() == [0, 0, 0]
