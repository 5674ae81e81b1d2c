"""How calls on a 4-bit cache use memory and take their arguments."""
import pytest
import torch

import differential_attention_05_b200 as da

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [None, torch.bfloat16, torch.float32])
def test_a_read_allocates_its_rows_and_nothing_else(packed, dtype):
    """New rows are the call's only allocations, at a length's first call as at the next."""
    cache = torch.zeros((2, 700, 3, 144), dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 300, 617], dtype=torch.int32, device="cuda")
    kw = dict(n_tokens=617, cu_seqlens=cu, max_seqlen=400) if packed else dict(n_tokens=617)
    size = 128 * 3 * 617 * (4 if dtype == torch.float32 else 2) * (1 if packed else 2)
    for _ in range(2):
        def count():
            s = torch.cuda.memory_stats()
            return s["allocation.all.allocated"], s["requested_bytes.all.allocated"]

        before = count()
        k, v = da.diffattn_kv4_read(cache, dtype=dtype, **kw)
        after = count()
        assert (after[0] - before[0], after[1] - before[1]) == (2, 2 * size)
        assert k.shape == v.shape == ((617, 3, 128) if packed else (2, 617, 3, 128))
        assert k.is_contiguous() and v.is_contiguous() and k.dtype == v.dtype == (dtype or torch.bfloat16)
        assert not k.any() and not v.any()


def test_counts_that_are_no_int32_are_refused():
    """None is cut to its low 32 bits: max_kv_len = 2^32 + 5 once meant 5 tokens."""
    big = (1 << 32) + 5
    pool = torch.zeros((4, 16, 2, 144), dtype=torch.uint8, device="cuda")
    table = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    lam = torch.zeros(2, device="cuda")
    k = torch.zeros((1, 7, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    for call in (
            lambda: da.diffattn_fwd_decode_kv4(q, pool, lam, block_table=table, max_kv_len=big),
            lambda: da.diffattn_fwd_decode_kv4(q, pool, lam, block_table=table, num_splits=big),
            lambda: da.diffattn_kv4_write(k, k, pool, block_table=table, max_kv_len=big),
            lambda: da.diffattn_kv4_write(k[0], k[0], pool, cu_seqlens=cu, max_seqlen=big, block_table=table),
            lambda: da.diffattn_kv4_write(k[:, :1].expand(1, big, 2, 128), k[:, :1].expand(1, big, 2, 128), pool,
                                          block_table=table),
            lambda: da.diffattn_kv4_read(pool, n_tokens=big, block_table=table)):
        with pytest.raises(da.DiffattnError):
            call()
