"""pa_blocks_step at the ends of what it takes: numbers of blocks that leave some lanes a last round of their own,
as many rows as there may be, tables near 2^31 entries."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import window_ref as wref
from .test_gpu_blocks import step
from .test_gpu_cache import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("back", [1, 31, 33, 511, 4095, 4097, 4096 + 511, 3 * 4096 + 17])
def test_blocks_given_back_that_fill_no_round(torch, back):
    """So many blocks of nine rows come back while a tenth row's are handed out, then with every third
    entry naming no block."""
    held = np.append(np.random.default_rng(back).multinomial(back, [1 / 9] * 9), 0)
    cols, blocks = int(held.max()) + 1, back + int(held.max()) + 1
    pool, want = pa.BlockPool.empty(10, cols, blocks, 16), wref.Pool(10, cols, blocks, 16)
    ctx, end = (16 * held).tolist(), [0] * 9 + [16 * cols]
    for _ in range(3):
        assert not step(torch, pool, want, ctx, ctx)
        assert not step(torch, pool, want, end, end)
    assert not step(torch, pool, want, ctx, ctx)
    spoiled = pool.block_tables.clone()
    lost = 0
    for b in range(9):
        spoiled[b, :held[b]:3] = blocks + b
        lost += -(-int(held[b]) // 3)
    pool.block_tables.copy_(spoiled)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.step(torch.zeros(10, dtype=torch.int32, device="cuda"), status=status)
    assert status.item() == pa.PA_STATUS_BIT_BLOCK_INDEX
    assert pool.count.item() == blocks and bool((pool.block_tables == -1).all())
    free = pool.free.tolist()
    assert free.count(-1) == lost and len(set(free) - {-1}) == blocks - lost


def test_as_many_entries_given_back_as_a_table_may_have(torch):
    """Rows that say that they hold every entry of a table of 2^31 - 2048, none of which names a block."""
    rows, cols, blocks = 2048, 2**20 - 1, 16
    tables = torch.full((rows, cols), -5, dtype=torch.int32, device="cuda")
    held = torch.full((rows,), cols, dtype=torch.int32, device="cuda")
    gone = torch.zeros_like(held)
    free = torch.full((blocks,), 7, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = pa.BlockPool(tables, held, gone, free, count, block_size=16)
    pool.step(torch.zeros_like(held))
    assert all(bool((part == -1).all()) for part in tables.split(64))
    assert bool((held == 0).all()) and count.item() == blocks and free.tolist() == [-1] * blocks
