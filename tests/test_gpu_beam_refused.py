"""PagedDecoder where a reordering or a fork is refused by the device: nothing of the requests changes, and later steps are right."""

import pytest
import torch

from tests.test_gpu_beam_decode import LAYERS, Model, chunk, decoder, step

pytestmark = pytest.mark.gpu
STATE = ("lens", "pos_offset", "free_head", "free_pages", "tables")


def begun(cuda, K, model, lens=(17, 40, 33, 50), offsets=(0, 5, 9, 2)):
    """Two sets of two beams with prompts of their own, whose texts were longer by `offsets`."""
    dec = decoder(cuda, K, 4, 160, 60, max_tokens=160, beams=2)
    dec.pos_offset.copy_(torch.tensor(offsets))
    chunk(dec, model, torch.arange(160, device=cuda), torch.tensor(lens, device=cuda))
    return dec


@pytest.mark.parametrize("what", ["parent", "page", "queue"])
@pytest.mark.parametrize("captured", [False, True])
def test_refused(cuda, what, captured):
    from attention_kv_cache_gb300 import kvsel as K
    model = Model(cuda, 3)
    dec, same = begun(cuda, K, model), begun(cuda, K, model)
    parents = torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device=cuda)
    good = parents.clone()
    keep, first = dec.free_head.clone(), dec.tables[3, 1].clone()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dec.reorder(parents)
    if what == "parent":
        parents[1, 0] = 2
    elif what == "page":
        dec.tables[3, 1] = 60
    else:
        dec.free_head.fill_(61)
    before = {x: getattr(dec, x).clone() for x in STATE}
    graph.replay() if captured else dec.reorder(parents)
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == (K.ERR_DEVICE if what == "page" else K.ERR_INVALID_ARG)
    for x in STATE:
        assert torch.equal(getattr(dec, x), before[x]), x
    # once what was wrong is put right, the same call and a step are those of a decoder that met no refusal
    dec.free_head.copy_(keep), dec.tables[3, 1].copy_(first), parents.copy_(good)
    graph.replay() if captured else dec.reorder(parents)
    same.reorder(good)
    tokens = torch.tensor([7, 8, 9, 10], device=cuda)
    assert torch.equal(step(dec, model, tokens), step(same, model, tokens))
    assert dec.pos_offset.tolist() == [5, 0, 2, 2] and dec.lens.tolist() == [41, 18, 51, 51]
    assert K.kvsel_read_device_error(dec.ws) == K.OK


def test_a_refused_fork_is_not_shared(cuda):
    """Beams that were not forked hold other pages: a layer reads each one's own."""
    from attention_kv_cache_gb300 import kvsel as K
    model = Model(cuda, 4)
    dec, same = begun(cuda, K, model), begun(cuda, K, model)
    head = dec.free_head.clone()
    dec.free_head.fill_(61)
    dec.fork()
    torch.cuda.synchronize()
    assert K.kvsel_read_device_error(dec.ws) == K.ERR_INVALID_ARG and dec.fork_rows.tolist() == [0, 0]
    dec.free_head.copy_(head)
    tokens = torch.tensor([7, 8, 9, 10], device=cuda)
    assert torch.equal(step(dec, model, tokens), step(same, model, tokens))
    assert K.kvsel_read_device_error(dec.ws) == K.OK and LAYERS == 2


def test_errors_of_a_step_captured_before_sharing(cuda):
    """Sharing needs more room than the captured step's workspace, in which its errors still arrive."""
    from attention_kv_cache_gb300 import kvsel as K
    model, tokens = Model(cuda), torch.tensor([1, 2, 3, 4], device=cuda)
    dec = decoder(cuda, K, 4, 64, 16)
    for _ in range(16):
        step(dec, model, tokens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(dec, model, tokens)
    small = dec.ws
    dec.share(torch.arange(5, device=cuda), torch.full((4,), 16, device=cuda))
    assert dec.ws is not small
    dec.free_head.fill_(16)                                    # no page is left for the next step's rows
    graph.replay()
    assert dec.device_error() == K.ERR_INVALID_ARG and dec.device_error() == K.OK
