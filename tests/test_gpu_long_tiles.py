"""Row tiles that take longer than a wait may: they are taken in segments, so that no wait is for all of one."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    yield torch
    pa.testing_set_wait_limit(0)


@pytest.mark.parametrize("call", ["window", "tree"])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("batch,q", [(4, 30), (1, 200)])
def test_row_tiles_longer_than_the_limit(torch, call, bits, batch, q):
    """32 row tiles of two million keys for all workers, some 6 ms each: most workers end one and begin another.
    The limit stands at 2 ms, twice what a segment of 65536 keys takes. Keys of zero, so
    that every weight is the same, values of 1 in three quarters of the blocks and -1 in the others:
    sums are of whole numbers below 2^24 (a power of two's multiples), so only the join of at most 152 parts
    (half a step each in the sums of weights and of values) and the result's rounding are off:
    2 * 152 * 2^-24 + 2^-12 < 3e-4 of 1/2 to 1."""
    bs, nb, d, H, Hk, keys = 128, 64, 64, 32, 8, 2**21
    cols, ones = keys // bs, keys // bs * 3 // 4
    g = torch.Generator(device="cuda").manual_seed(q)
    dtype = torch.float16 if bits == 16 else torch.float8_e4m3fn
    key = torch.zeros((nb, bs, Hk, d), device="cuda").to(dtype)
    value = torch.ones((nb, bs, Hk, d), device="cuda")
    value[nb // 2:] = -1
    exps = [None, None]
    if bits == 8:
        exps = [torch.full((nb, Hk, bs), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    tables = torch.randint(0, nb // 2, (batch, cols), generator=g, device="cuda", dtype=torch.int32)
    tables[:, ones:] += nb // 2
    lens, qs = (torch.full((batch,), n, dtype=torch.int32, device="cuda") for n in (keys, q))
    query = torch.ones((batch * q, H, d), dtype=torch.float16, device="cuda")
    out = torch.full_like(query, 7.0)
    shape = dict(batch=batch, num_heads=H, max_seqlen_q=q, max_blocks_per_seq=cols)
    if call == "window":
        step = pa.WindowStep(key, value.to(dtype), *exps, **shape, window=2**31 - 1)
        run = lambda: step.run(query, tables, lens, qs, out)  # noqa: E731
    else:
        step = pa.TreeStep(key, value.to(dtype), *exps, **shape)
        run = lambda: step.run(query, tables, lens, qs, None, out)  # noqa: E731
    pa.testing_set_wait_limit(2**22)
    try:
        run()
        assert step.status() == (pa.PA_OK, 0)
    finally:
        pa.testing_set_wait_limit(0)
    seen = keys - q + 1 + np.arange(q)
    want = np.tile((2.0 * ones * bs - seen) / seen, batch)
    assert np.abs(out.cpu().numpy().astype(np.float64) - want[:, None, None]).max() < 3e-4
