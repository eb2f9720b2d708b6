"""What a pool's binding refuses before its sizes are cut to 32 bits."""
import pytest
import torch

import paged_kv_cache_206_gb300 as pa


def ints(*shape):
    return torch.empty(shape, dtype=torch.int32, device="meta")  # (shapes alone)


@pytest.mark.parametrize("batch,cols,blocks", [(2, 4, 2**32 + 6), (2, 2**32 + 4, 6), (2**32 + 2, 4, 6), (2, 4, 2**31)])
def test_a_pool_of_more_than_32_bits_is_refused(batch, cols, blocks):
    with pytest.raises(pa.PaError) as e:
        pa.BlockPool(ints(batch, cols), ints(batch), ints(batch), ints(blocks), ints(1), block_size=16)
    assert e.value.status == pa.PA_ERR_INVALID_ARG and "2^31" in str(e.value)
