"""Waits of the tree attention kernels that run out, without a GPU fault: with a limit of a few cycles
a correct launch must report PA_ERR_TIMEOUT, exit with its copies landed and its tensor memory
freed, and leave the context usable: with the default limit back the same call gives the same bits."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from .test_gpu_tree import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    yield torch
    pa.testing_set_wait_limit(0)


# drafts, H, Hk, dims: up to 8 and 16 rows of a kv head (warp-level instructions), up to 128 and more (tcgen05);
# full batches of long contexts, so that memory is what the kernels wait for
CASES = [(1, 32, 8, 128), (4, 32, 8, 128), (2, 16, 4, 256), (16, 32, 8, 128), (16, 32, 8, 64), (64, 32, 8, 128)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_short_wait_limit_times_out_and_the_context_survives(torch, bits, case):
    drafts, H, Hk, d = case
    B, bs = 24, 64
    rng = np.random.default_rng(drafts)
    g = torch.Generator(device="cuda").manual_seed(drafts)
    q = rng.integers(max(1, drafts // 2), drafts + 1, B).astype(np.int32)
    ctx = np.maximum(q, rng.integers(64, 8193, B)).astype(np.int32)
    need = -(-ctx // bs)
    tables = np.full((B, int(need.max())), -1, np.int32)
    ids = rng.permutation(int(need.sum())).astype(np.int32)
    for b in range(B):
        tables[b, :need[b]] = ids[need[:b].sum():need[:b + 1].sum()]
    k, v = (torch.randn((len(ids), bs, Hk, d), generator=g, device="cuda").half() for _ in range(2))
    exps = [None, None]
    if bits == 8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        exps = [torch.randint(125, 129, (len(ids), Hk, bs), generator=g, device="cuda").to(torch.uint8)
                for _ in range(2)]
    query = torch.randn((int(q.sum()), H, d), generator=g, device="cuda").half()
    step = pa.TreeStep(k, v, *exps, batch=B, num_heads=H, max_seqlen_q=drafts,
                       max_blocks_per_seq=tables.shape[1])
    args = (query, up(torch, tables), up(torch, ctx), up(torch, q), up(torch, ref.trees(rng, q, "tree")),
            torch.empty_like(query))
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    first = step.run(*args).clone()
    assert step.status() == (pa.PA_OK, 0)
    # whether a wait outlasts 32 cycles depends on when its copy lands: from HBM, in three tries
    for _ in range(3):
        flush.zero_()
        pa.testing_set_wait_limit(32)
        try:
            step.run(*args)
            st, word = step.status()
        finally:
            pa.testing_set_wait_limit(0)
        if st == pa.PA_ERR_TIMEOUT:
            break
    assert st == pa.PA_ERR_TIMEOUT and word == pa.PA_STATUS_BIT_TIMEOUT
    pa.pa_status_clear(step.workspace)
    for _ in range(3):
        assert torch.equal(step.run(*args), first)
    assert step.status() == (pa.PA_OK, 0)
