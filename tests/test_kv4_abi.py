"""Refusals of the 4-bit KV cache's entry points, on the host: nothing here needs a GPU."""
import ctypes

import pytest
import torch

import differential_attention_05_b200 as da
from differential_attention_05_b200 import _binding as B

GOOD = 0x10000
vp = ctypes.c_void_p
REC = 144


@pytest.fixture(scope="module")
def lib():
    return da.load_library()


def _rows(**kw):
    p = B.Kv4Rows()
    p.dtype, p.batch, p.n_tokens, p.max_seqlen, p.n_kv_heads, p.max_kv_len = B.DIFFATTN_BF16, 2, 16, 0, 4, 64
    p.k_strides[:] = p.v_strides[:] = (16 * 4 * 128, 4 * 128, 128)
    p.cache_strides[:] = (64 * 4 * REC, 4 * REC, REC)
    for n, v in kw.items():
        if n.endswith("strides"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    return p


def _pool(**kw):
    pk = B.PagedKV()
    pk.page_size, pk.num_pages, pk.max_pages_per_seq = 16, 10, 4
    pk.page_strides[:] = (16 * 4 * REC, 4 * REC, REC)
    for n, v in kw.items():
        if n.endswith("strides"):
            getattr(pk, n)[:] = v
        else:
            setattr(pk, n, v)
    return pk


def _write(lib, p, pk=None, k=GOOD, v=GOOD, cu=None, pos=None, cache=GOOD, table=None):
    return lib.diffattn_kv4_write(None if p is None else ctypes.byref(p), None if pk is None else ctypes.byref(pk),
                                  vp(k), vp(v), vp(cu), vp(pos), vp(cache), vp(table), None, None)


def _read(lib, p, pk=None, k=GOOD, v=GOOD, cu=None, pos=None, cache=GOOD, table=None):
    return lib.diffattn_kv4_read(None if p is None else ctypes.byref(p), None if pk is None else ctypes.byref(pk),
                                 vp(cache), vp(table), vp(cu), vp(pos), vp(k), vp(v), None, None)


ROWS = [(dict(dtype=2), -1), (dict(batch=-1), -1), (dict(n_tokens=-1), -1), (dict(n_kv_heads=0), -1),
        (dict(max_kv_len=-1), -1), (dict(batch=65536), -2), (dict(max_kv_len=(1 << 30) + 1), -2),
        (dict(n_kv_heads=65536), -2), (dict(n_tokens=(1 << 31) - 1, n_kv_heads=65535), -2),
        (dict(k_strides=(-8, 512, 128)), -1), (dict(v_strides=(8192, 512, -128)), -1),
        (dict(k_strides=(8192, 512, 4)), -3), (dict(v_strides=(8196, 512, 128)), -3),
        (dict(dtype=B.DIFFATTN_F32, k_strides=(8192, 514, 128)), -3),
        (dict(cache_strides=(64 * 4 * REC, 4 * REC, 128)), -1), (dict(cache_strides=(64 * 4 * REC, 0, REC)), -1),
        (dict(cache_strides=(0, 4 * REC, REC)), -1), (dict(cache_strides=(64 * 4 * REC, 4 * REC, REC + 8)), -3),
        (dict(cache_strides=(-16, 4 * REC, REC)), -1)]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,code", ROWS)
def test_rows_refused(lib, call, kw, code):
    assert call(lib, _rows(**kw)) == code


@pytest.mark.parametrize("call", [_write, _read])
def test_rows_pointers(lib, call):
    assert call(lib, None) == -1
    for name in ("k", "v", "cache"):
        assert call(lib, _rows(), **{name: None}) == -1
        assert call(lib, _rows(), **{name: GOOD + 8}) == -3
    assert call(lib, _rows(), _pool()) == -1  # no block table
    assert call(lib, _rows(max_seqlen=-1), cu=GOOD) == -1
    # nothing to move: no pointer is needed
    for kw in (dict(batch=0), dict(n_tokens=0)):
        assert call(lib, _rows(**kw), k=None, v=None, cache=None) == 0
    assert call(lib, _rows(max_seqlen=0), cu=GOOD, k=None, v=None, cache=None) == 0


POOLS = [(dict(page_size=0), -1), (dict(page_size=12), -1), (dict(page_size=1 << 17), -1), (dict(num_pages=0), -1),
         (dict(max_pages_per_seq=0), -1), (dict(max_pages_per_seq=3), -1), (dict(reserved=1), -1),
         (dict(page_strides=(16 * 4 * REC, 4 * REC, 16)), -1), (dict(page_strides=(16 * 4 * REC, 4 * REC + 4, REC)), -3),
         (dict(page_strides=(0, 4 * REC, REC)), -1)]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,code", POOLS)
def test_pools_refused(lib, call, kw, code):
    assert call(lib, _rows(), _pool(**kw), table=GOOD) == code


def _params(variant=2, **kw):
    p = B.DecodeParams()
    p.variant, p.dtype, p.batch, p.max_kv_len = variant, B.DIFFATTN_BF16, 2, 64
    p.n_q_heads, p.n_kv_heads, p.head_dim, p.num_splits = (16, 4, 128, 0) if variant == 2 else (4, 4, 64, 0)
    p.q_strides[:] = (p.n_q_heads * 128, 128)
    p.kv_strides[:] = (64 * 4 * REC, 4 * REC, REC)
    p.o_strides[:] = (8 * 128, 128)
    for n, v in kw.items():
        if n.endswith("strides"):
            getattr(p, n)[:] = v
        else:
            setattr(p, n, v)
    return p


def _decode(lib, p, pk=None, q=GOOD, cache=GOOD, table=None, lam=GOOD, li=None, norm=0, eps=1e-5, out=GOOD, ws=GOOD,
            ws_bytes=1 << 30):
    return lib.diffattn_fwd_decode_kv4(None if p is None else ctypes.byref(p), None if pk is None else ctypes.byref(pk),
                                       vp(q), vp(cache), vp(table), None, vp(lam), vp(li), norm, eps, vp(out), vp(ws),
                                       ws_bytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(variant=3), -1), (dict(dtype=B.DIFFATTN_F32), -2), (dict(dtype=7), -1), (dict(batch=-1), -1),
    (dict(max_kv_len=-1), -1), (dict(n_q_heads=10), -1), (dict(n_q_heads=4), -1), (dict(head_dim=64), -2),
    (dict(num_splits=-1), -1), (dict(batch=65536), -2), (dict(max_kv_len=(1 << 30) + 1), -2),
    (dict(q_strides=(-8, 128)), -1), (dict(q_strides=(2048, 130)), -3), (dict(o_strides=(1024, 4)), -3),
    (dict(kv_strides=(64 * 4 * REC, 4 * REC, 16)), -1), (dict(kv_strides=(64 * 4 * REC, 4 * REC, REC + 1)), -3)])
def test_decode_refused(lib, kw, code):
    assert _decode(lib, _params(**kw)) == code


def test_decode_pointers_norm_and_workspace(lib):
    assert _decode(lib, None) == -1
    for name in ("q", "cache", "lam", "out"):
        assert _decode(lib, _params(), **{name: None}) == -1
    for name in ("q", "cache", "out"):
        assert _decode(lib, _params(), **{name: GOOD + 2}) == -3
    assert _decode(lib, _params(), norm=1, li=GOOD) == -1  # V2 has no norm
    assert _decode(lib, _params(), norm=2) == -1
    assert _decode(lib, _params(1), norm=1) == -1  # V1's norm needs lambda_init
    assert _decode(lib, _params(1), norm=1, li=GOOD, eps=-1.0) == -1
    assert _decode(lib, _params(1), norm=1, li=GOOD, eps=float("nan")) == -1
    assert _decode(lib, _params(1, n_q_heads=8)) == -1
    assert _decode(lib, _params(), _pool()) == -1
    for kw, code in POOLS:
        assert _decode(lib, _params(), _pool(**kw), table=GOOD) == code
    # the workspace: two units' states of every block, 4 heads of 8 rows each here
    n = ctypes.c_size_t(1)
    size = lib.diffattn_decode_kv4_workspace_size
    for splits, L, blocks in ((1, 1000, 2), (3, 1000, 6), (0, 1000, 32), (0, 128, 0), (0, 129, 5), (9, 64, 4), (2, 0, 1)):
        p = _params(num_splits=splits, max_kv_len=L, kv_strides=(1000 * 4 * REC, 4 * REC, REC))
        assert size(ctypes.byref(p), None, ctypes.byref(n)) == 0
        assert n.value == blocks * 2 * 4 * 8 * 130 * 4, (splits, L)
    p = _params(max_kv_len=1 << 20, kv_strides=(4 * REC << 20, 4 * REC, REC), n_q_heads=64)
    assert size(ctypes.byref(p), None, ctypes.byref(n)) == 0 and n.value < 20 << 20
    # the layout takes part: heads that do not lie side by side go one to a block
    p = _params(max_kv_len=2048, n_q_heads=16)
    pk = _pool(max_pages_per_seq=128)
    assert size(ctypes.byref(p), ctypes.byref(pk), ctypes.byref(n)) == 0
    assert n.value == 64 * 2 * 4 * 8 * 130 * 4
    apart = _pool(max_pages_per_seq=128, page_strides=(16 * 4 * 160, 4 * 160, 160))
    assert size(ctypes.byref(p), ctypes.byref(apart), ctypes.byref(n)) == 0
    assert n.value == 16 * 4 * 2 * 1 * 8 * 130 * 4
    # short entries need none
    assert _decode(lib, _params(batch=0), ws=None) == 0
    p = _params(max_kv_len=2048, kv_strides=(2048 * 4 * REC, 4 * REC, REC))
    assert size(ctypes.byref(p), None, ctypes.byref(n)) == 0
    assert _decode(lib, p, ws=None) == -4
    assert _decode(lib, p, ws_bytes=n.value - 1) == -4
    assert _decode(lib, p, ws=GOOD + 16) == -3
    assert size(ctypes.byref(p), None, None) == -1
    assert _decode(lib, _params(batch=0), q=None, cache=None, lam=None, out=None, ws=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    cache = torch.zeros((1, 4, 2, 144), dtype=torch.uint8)
    k = torch.zeros((1, 4, 2, 128), dtype=torch.bfloat16)
    for bad in (cache, cache.int(), cache[..., :128]):
        with pytest.raises(da.DiffattnError):
            da.diffattn_kv4_write(k, k, bad)
    for kk, vv in ((k.half(), k.half()), (k, k.float()), (k[..., :64], k), (k, k[:, :2]), (k[..., ::2], k)):
        with pytest.raises(da.DiffattnError):
            da.diffattn_kv4_write(kk, vv, cache)
    assert da.KV4_RECORD_BYTES == B.KV4_RECORD_BYTES == 144
