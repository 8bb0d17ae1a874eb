"""What the tests of the paged calls share: pools of any layout, block tables, workspaces."""

from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def kinds(K):
    return {"bf16": K.DTYPE_BF16, "f16": K.DTYPE_F16, "e4m3": K.DTYPE_E4M3}


def workspace(K, n, cuda):
    buf = torch.zeros(n + K.WS_ALIGN, dtype=torch.uint8, device=cuda)
    off = (-buf.data_ptr()) % K.WS_ALIGN
    return buf[off:off + n]


def blocks_of(lens, P, max_blocks, n_pages, rng, fill=-7):
    """Block tables [batch, max_blocks] of distinct random pages; entries behind a request's last page are `fill`."""
    ids = rng.permutation(n_pages)
    tables = np.full((len(lens), max_blocks), fill, np.int64)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // P)
        tables[b, :m] = ids[at:at + m]
        at += m
    return tables


def pool_view(pool, order):
    """[page, row, head, d] view of a pool."""
    return pool if order == "row" else pool.transpose(1, 2)


def empty_pool(n_pages, P, h_kv, d, order, dtype, device, nan=True):
    """A pool whose every row is NaN (or zero)."""
    shape = (n_pages, h_kv, P, d) if order == "head" else (n_pages, P, h_kv, d)
    if dtype == torch.float8_e4m3fn:
        return torch.full(shape, 0x7f if nan else 0, dtype=torch.uint8, device=device).view(dtype)
    return torch.full(shape, float("nan") if nan else 0.0, dtype=dtype, device=device)


def put_rows(pool, order, tables, P, b, first, rows):
    """rows [n, h_kv, d] as rows first .. of request b."""
    if rows.shape[0] == 0:
        return
    t = torch.arange(first, first + rows.shape[0])
    page = torch.as_tensor(tables[b], dtype=torch.int64)[t // P].to(pool.device)
    view = pool_view(pool, order)
    if pool.element_size() == 1:
        view, rows = pool_view(pool.view(torch.uint8), order), rows.view(torch.uint8)
    view[page, (t % P).to(pool.device)] = rows.to(pool.device)


def f64(t):
    return t.detach().float().cpu().double().numpy()
