"""Sums over a million keys by the kernel of heads above 256 dims: one that adds the keys one by one in fp32
loses 0.3 % of these, eight steps of the fp16 result."""
import math

import pytest

import paged_kv_cache_206_gb300 as pa

pytestmark = pytest.mark.gpu

KEYS, BLOCK, DIM = 2**20, 128, 272


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


def attend(torch, call, bits, key, value, tables):
    """One token at the end of KEYS keys; the caches' blocks hold numbers that both types hold exactly."""
    exps = [None, None]
    dtype = torch.float16
    if bits == 8:
        dtype = torch.float8_e4m3fn
        exps = [torch.full((key.shape[0], 1, BLOCK), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    shape = dict(batch=1, num_heads=1, max_seqlen_q=1, max_blocks_per_seq=tables.shape[1], scale=1.0)
    caches = key.to(dtype), value.to(dtype), *exps
    query = torch.zeros((1, 1, DIM), dtype=torch.float16, device="cuda")
    query[..., 0] = 1
    out = torch.full_like(query, 7.0)
    lens = torch.tensor([KEYS], dtype=torch.int32, device="cuda")
    if call == "window":
        step = pa.WindowStep(*caches, **shape, window=2**31 - 1)
        step.run(query, tables, lens, None, out)
    else:
        step = pa.TreeStep(*caches, **shape)
        step.run(query, tables, lens, None, None, out)
    assert step.status() == (pa.PA_OK, 0)
    return out[0, 0].double().cpu()


@pytest.mark.parametrize("call", ["window", "tree"])
def test_values_of_equal_weights(torch, call):
    """Equal scores over equal values 1 + 2^-7 are that value: sums that are off by less than 2^-13 of it
    (an element's half step is 2^-12) round to it."""
    key = torch.zeros((1, BLOCK, 1, DIM), device="cuda")
    value = torch.full_like(key, 1 + 2.0**-7)
    tables = torch.zeros((1, KEYS // BLOCK), dtype=torch.int32, device="cuda")
    assert bool((attend(torch, call, 16, key, value, tables) == 1 + 2.0**-7).all())


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("call", ["window", "tree"])
def test_the_sum_of_weights(torch, call, bits):
    """Four keys of score 0 (one for each of four that take turns), all others of -0.75; values of 1 in a sixteenth
    of the blocks, 0 behind them. Fewer than 2^7 roundings in a row (2^-17) and the result's (2^-11)."""
    key = torch.zeros((3, BLOCK, 1, DIM), device="cuda")
    key[..., 0] = -0.75
    key[0, :4] = 0
    value = torch.zeros_like(key)
    value[:2] = 1
    ones = KEYS // BLOCK // 16
    tables = torch.full((1, KEYS // BLOCK), 2, dtype=torch.int32, device="cuda")
    tables[0, :ones] = 1
    tables[0, 0] = 0
    w = math.exp(-0.75)
    want = (4 + (ones * BLOCK - 4) * w) / (4 + (KEYS - 4) * w)
    got = attend(torch, call, bits, key, value, tables)
    assert bool(((got - want).abs() <= (2.0**-11 + 2.0**-16) * want).all())
