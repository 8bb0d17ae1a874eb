"""Beams that share their prompt's rows and beams that read their own, fed the same tokens and parents: the same pools, and every
layer's output of every step within the two calls' tolerances of the other's.

Each call's output is within half a step of its value (2^-8 in bf16), and of a mean of |v| m by its scores' and weights' errors: 2 dz + ...
below 2^-13 m over a bf16 pool, and below 2^-13 m + 2^-11 m (a shared row's weight rounded once to fp16) over an e4m3 one; rows of V are
standard normals (or such rounded to 8 bits), whose m is below 2.  So two of them differ by 2^-7 |o| + 2^-11, or 2^-7 |o| + 2^-9, at most.
"""

import pytest
import torch

from tests.test_gpu_beam_decode import HKV, LAYERS, VOCAB, Model, chunk, decoder, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_dtype", [None, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_shared_rows_change_nothing(cuda, cache_dtype, captured):
    from attention_kv_cache_gb300 import kvsel as K
    sets, beams, model, g = 2, 4, Model(cuda, 8), torch.Generator().manual_seed(4)
    batch = sets * beams
    scales = None if cache_dtype is None else tuple((0.02 + torch.zeros(LAYERS, HKV)).to(cuda) for _ in range(2))
    text = torch.randint(0, VOCAB, (140,), generator=g).to(cuda)
    n_new = torch.zeros(batch, dtype=torch.int64, device=cuda)
    n_new[::beams] = torch.tensor([50, 90], device=cuda)
    plan = [(torch.randint(0, VOCAB, (batch,), generator=g).to(cuda), torch.randint(0, beams, (sets, beams), generator=g).int().to(cuda))
            for _ in range(24)]
    decs, outs, graphs = [], [], []
    now, parents = plan[0][0].clone(), plan[0][1].clone()
    for shared in (True, False):
        dec = decoder(cuda, K, batch, 160, 100, max_tokens=140, beams=beams, cache_dtype=cache_dtype, scales=scales)
        chunk(dec, model, text, n_new)
        dec.fork()
        assert dec.fork_rows.tolist() == [48, 80]
        if not shared:
            dec.share(None, None)
        out = torch.empty((batch, LAYERS, *dec.o.shape[1:]), dtype=dec.o.dtype, device=cuda)

        def one(dec=dec, out=out):
            out.copy_(step(dec, model, now))
            dec.reorder(parents)

        if captured:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                one()
        else:
            graphs.append(one)
        decs.append(dec)
        outs.append(out)
    slack = 2.0 ** -11 if cache_dtype is None else 2.0 ** -9
    for i, (tokens, chosen) in enumerate(plan):
        now.copy_(tokens), parents.copy_(chosen)
        for run in graphs:
            run.replay() if captured else run()
        a, b = (x.float() for x in outs)
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + slack).all(), (i, (a - b).abs().max())
        assert not torch.equal(a, torch.zeros_like(a))
    for x in ("lens", "free_head", "free_pages", "pos_offset"):
        assert torch.equal(getattr(decs[0], x), getattr(decs[1], x)), x
    for t0, t1, n in zip(decs[0].tables, decs[1].tables, decs[0].lens.tolist()):
        assert torch.equal(t0[:-(-n // 16)], t1[:-(-n // 16)])
    assert all(d.device_error() == K.OK for d in decs)
