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


def test_captured_behind_work_of_another_stream():
    """A write whose rows another stream makes, captured with that stream's work, a copy and the
    calls that read the cache: every replay follows the inputs."""
    B, H, L = 2, 4, 500
    gen = torch.Generator(device="cuda").manual_seed(3)
    src = torch.randn((2, B, 64, H, 128), generator=gen, device="cuda").bfloat16()
    rows = torch.zeros_like(src)
    cache = torch.zeros((B, L, H, 144), dtype=torch.uint8, device="cuda")
    q = torch.randn((B, 8 * H, 128), generator=gen, device="cuda").bfloat16()
    lam = torch.full((4 * H,), 0.7, device="cuda")
    at, length = torch.zeros((2, B), dtype=torch.int32, device="cuda")
    length += 64
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            rows[0].copy_(src[0] * 2)
        rows[1].copy_(src[1])
        main.wait_stream(side)
        da.diffattn_kv4_write(rows[0], rows[1], cache, pos=at)
        out = da.diffattn_fwd_decode_kv4(q, cache, lam, kv_len=length)
        long = da.diffattn_fwd_decode_kv4(q, cache, lam, kv_len=length, num_splits=3)
        k, v = da.diffattn_kv4_read(cache, n_tokens=64, pos=at)
        at.add_(1)
        length.add_(1)
        return out, long, k, v

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        want = [[t.clone() for t in step()]]
        for _ in range(3):
            src.neg_()
            want.append([t.clone() for t in step()])
    main.synchronize()
    src.neg_()  # four sign changes in all
    at.zero_()
    length.fill_(64)
    cache.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        outs = step()
    at.zero_()
    length.fill_(64)
    cache.zero_()
    torch.cuda.synchronize()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i
        src.neg_()
        torch.cuda.synchronize()
