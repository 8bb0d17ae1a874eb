"""PagedDecoder: prompts that replace others behind a fork, without a fork of their own."""

import pytest
import torch

from tests.test_gpu_beam_decode import D, HKV, LAYERS, VOCAB, Model, chunk, decoder, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["chunk", "captured chunk", "admit"])
def test_every_beam_reads_its_own_rows(cuda, way):
    from attention_kv_cache_gb300 import kvsel as K
    model, n = Model(cuda, 6), [110, 130, 97, 120]
    g = torch.Generator().manual_seed(1)
    text = torch.randint(0, VOCAB, (480,), generator=g).to(cuda)
    held = [torch.randn(4, LAYERS, HKV, 100, D, generator=g).bfloat16().to(cuda) for _ in range(2)]
    rows, tokens = torch.tensor(n, device=cuda), torch.tensor([1, 2, 3, 4], device=cuda)
    outs = []
    for forked in (True, False):
        dec = decoder(cuda, K, 4, 160, 60, max_tokens=480, beams=2)

        def come():
            if way == "admit":
                dec.admit(*held, [100] * 4)
            else:
                chunk(dec, model, text, rows)

        if way == "captured chunk":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                come()
        if forked:
            chunk(dec, model, torch.arange(480, device=cuda), torch.tensor([100, 0, 96, 0], device=cuda))
            dec.fork()
            dec.lens.zero_(), dec.free_head.zero_()
            dec.free_pages.copy_(torch.arange(60, dtype=torch.int32, device=cuda))
        graph.replay() if way == "captured chunk" else come()
        outs.append(step(dec, model, tokens))
        assert dec.device_error() == K.OK
    assert torch.equal(*outs)
