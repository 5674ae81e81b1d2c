"""The KV cache held in 4 bits on the GPU: rows written into it and read back, against the
format's definition in 64 bits (records equal byte for byte, values equal), and the decode
over it against plain 64-bit attention over the cache's values, within the roundings' bound
(kv4_plain.decode)."""
import numpy as np
import pytest
import torch

import differential_attention_05_b200 as da

import kv4_plain as plain

pytestmark = pytest.mark.gpu

SENTINEL = 0xAB


def _rng(seed):
    return np.random.default_rng(seed)


def _rows(rng, shape, dtype, scale=1.0):
    """Device rows and the bf16 values the cache sees of them (float64)."""
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    if dtype == torch.bfloat16:
        x = plain.bf16_round(x).astype(np.float32)
    return torch.from_numpy(x).cuda().to(dtype), plain.bf16_round(x)


def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


class Cache:
    """A cache of B entries with L positions and H heads, contiguous (page = 0) or paged in a
    shuffled pool with spare pages, every byte SENTINEL at first."""

    def __init__(self, B, L, H, page=0, seed=0, head_major=False):
        self.B, self.L, self.H, self.page = B, L, H, page
        if page:
            each = -(-L // page)
            self.pool = B * each + 2
            self.table = torch.from_numpy(
                _rng(seed).permutation(self.pool)[:B * each].reshape(B, each).astype(np.int32)).cuda()
            lead = (self.pool, page)
        else:
            self.table, lead = None, (B, L)
        if head_major:
            self.t = torch.full((lead[0], H, lead[1], 144), SENTINEL, dtype=torch.uint8, device="cuda").transpose(1, 2)
        else:
            self.t = torch.full((*lead, H, 144), SENTINEL, dtype=torch.uint8, device="cuda")

    @property
    def where(self):
        return dict(block_table=self.table, max_kv_len=self.L)

    def entries(self):
        """[B, L, H, 144] bytes on the host."""
        t = self.t.cpu().numpy()
        if self.table is None:
            return t
        return t[self.table.cpu().numpy()].reshape(self.B, -1, self.H, 144)[:, :self.L]

    def set_entries(self, rec):
        rec = torch.from_numpy(np.ascontiguousarray(rec)).cuda()
        if self.table is None:
            self.t.copy_(rec)
            return self
        pad = self.table.shape[1] * self.page - self.L
        rec = torch.cat((rec, torch.full_like(rec[:, :1], 0xFF).expand(-1, pad, -1, -1)), 1)
        self.t[self.table.long()] = rec.view(self.B, -1, self.page, self.H, 144)
        return self


def _cu(lens):
    return _i32(np.concatenate(([0], np.cumsum(lens))))


# ---- writing and reading --------------------------------------------------------------

@pytest.mark.parametrize("page", [0, 1, 2, 16, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,N,pos", [(1, 1, None), (3, 33, (5, 0)), (8, 70, (0, 11)), (2, 1, (80, 3))])
def test_write_and_read_fixed_length(page, dtype, H, N, pos):
    B, L = 2, 81
    rng = _rng(page + H)
    c = Cache(B, L, H, page, seed=H)
    before = c.entries()
    k, kx = _rows(rng, (B, N, H, 128), dtype)
    v, vx = _rows(rng, (B, N, H, 128), dtype, 3.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = None if pos is None else _i32(pos)
    assert da.diffattn_kv4_write(k, v, c.t, pos=p, dev_status=st, **c.where) is c.t
    want = before.copy()
    for b in range(B):
        at = 0 if pos is None else pos[b]
        want[b, at:at + N] = plain.records(kx[b], vx[b])
    assert np.array_equal(c.entries(), want)
    kb, vb = da.diffattn_kv4_read(c.t, n_tokens=N, pos=p, dtype=dtype, dev_status=st, **c.where)
    for b in range(B):
        at = 0 if pos is None else pos[b]
        for got, ref in zip((kb[b], vb[b]), plain.values(want[b, at:at + N])):
            ref = plain.bf16_round(ref) if dtype == torch.bfloat16 else ref
            assert np.array_equal(got.double().cpu().numpy(), ref)
    assert st.item() == 0
    if page:  # nothing but the entries' rows was touched
        used = torch.zeros(c.t.shape[:2], dtype=torch.bool, device="cuda")
        for b in range(B):
            at = 0 if pos is None else pos[b]
            for t in range(at, at + N):
                used[c.table[b, t // page].long(), t % page] = True
        assert (c.t[~used] == SENTINEL).all()


@pytest.mark.parametrize("page", [0, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_and_read_packed(page, dtype):
    lens, pos, H, L = [7, 0, 65, 1, 33], [0, 3, 10, 74, 40], 3, 75
    rng = _rng(31)
    total = sum(lens) + 4  # four rows that no entry owns
    c = Cache(5, L, H, page, seed=3)
    want = c.entries().copy()
    k, kx = _rows(rng, (total, H, 128), dtype)
    v, vx = _rows(rng, (total, H, 128), dtype)
    cu, p = _cu(lens), _i32(pos)
    da.diffattn_kv4_write(k, v, c.t, pos=p, cu_seqlens=cu, max_seqlen=65, **c.where)
    row = 0
    for b, n in enumerate(lens):
        want[b, pos[b]:pos[b] + n] = plain.records(kx[row:row + n], vx[row:row + n])
        row += n
    assert np.array_equal(c.entries(), want)
    kb, vb = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    da.diffattn_kv4_read(c.t, pos=p, cu_seqlens=cu, max_seqlen=70, k=kb, v=vb, **c.where)
    rk, rv = plain.values(plain.records(kx, vx))
    for got, ref in ((kb, rk), (vb, rv)):
        ref = plain.bf16_round(ref) if dtype == torch.bfloat16 else ref
        assert np.array_equal(got[:-4].double().cpu().numpy(), ref[:-4])
        assert (got[-4:] == 7.0).all()


def test_packed_rows_under_the_largest_max_seqlen():
    """A caller that knows no better bound than int32's may give that one: the rows of the tensors
    bound the launch. New rows of a read have the cache's heads and the type asked for."""
    lens, H = [3, 0, 9], 2
    rng = _rng(32)
    c = Cache(3, 12, H, 4, seed=4)
    want = c.entries().copy()
    k, kx = _rows(rng, (12, H, 128), torch.bfloat16)
    v, vx = _rows(rng, (12, H, 128), torch.bfloat16)
    cu = _cu(lens)
    da.diffattn_kv4_write(k, v, c.t, cu_seqlens=cu, max_seqlen=2**31 - 1, **c.where)
    row = 0
    for b, n in enumerate(lens):
        want[b, :n] = plain.records(kx[row:row + n], vx[row:row + n])
        row += n
    assert np.array_equal(c.entries(), want)
    rk, rv = plain.values(plain.records(kx, vx))
    for dtype in (None, torch.float32):
        for _ in range(2):  # the second call finds the first one's plan
            got = da.diffattn_kv4_read(c.t, n_tokens=12, cu_seqlens=cu, max_seqlen=2**31 - 1, dtype=dtype, **c.where)
            for x, ref in zip(got, (rk, rv)):
                assert x.dtype == (dtype or torch.bfloat16) and x.shape == (12, H, 128) and x.is_contiguous()
                ref = plain.bf16_round(ref) if dtype is None else ref
                assert np.array_equal(x.double().cpu().numpy(), ref)
            assert got[0].data_ptr() != got[1].data_ptr()


def test_special_groups():
    """Zeros of both signs, +-ties, a lone element, NaN, infinities, the type's extremes,
    subnormals, values around the zero threshold, and ties between codes."""
    x = np.zeros((1, 12, 1, 128), dtype=np.float32)
    x[0, 0, 0, :32] = -0.0
    x[0, 1, 0, [0, 1]] = [2.0, -2.0]
    x[0, 1, 0, 40] = 3.0
    x[0, 2, 0, [3, 70]] = [np.nan, np.inf]
    x[0, 2, 0, 100] = -np.inf
    big = float(torch.finfo(torch.bfloat16).max)
    x[0, 3, 0, :64] = np.linspace(-big, big, 64)
    x[0, 4, 0, :128] = np.linspace(-1, 1, 128) * 1e-39
    x[0, 5, 0, [0, 32, 64, 96]] = [2.0 ** -100, 2.0 ** -101, -2.0 ** -100, 1.5 * 2.0 ** -101]
    x[0, 6, 0, :32] = np.arange(32) * 0.5 - 8  # scale 1, every code and every tie
    x[0, 7, 0, :32] = 8 - np.arange(32) * 0.5  # scale -1
    x[0, 8, 0] = 1.0
    x[0, 9, 0] = -1.0
    x[0, 10, 0] = np.where(np.arange(128) % 2, 7.75, -8.0)
    x[0, 11, 0] = np.exp2(np.linspace(-30, 5, 128)) * np.where(np.arange(128) % 3, 1, -1)
    for dtype in (torch.bfloat16, torch.float32):
        k = torch.from_numpy(x).cuda().to(dtype)
        v = k.flip(1).contiguous()
        c = Cache(1, 12, 1)
        da.diffattn_kv4_write(k, v, c.t)
        kx = k.bfloat16().double().cpu().numpy()
        want = plain.records(kx, v.bfloat16().double().cpu().numpy())
        assert np.array_equal(c.entries(), want)
        kb, vb = da.diffattn_kv4_read(c.t, n_tokens=12, dtype=torch.float32)
        rk, rv = plain.values(want)
        np.testing.assert_array_equal(kb.double().cpu().numpy(), rk)
        np.testing.assert_array_equal(vb.double().cpu().numpy(), rv)


def test_every_quotient_of_significands():
    """All 128 significands of a group's largest element, of either sign, against every bf16
    value from 2^-6 of it upwards: codes equal to exact rounding of the quotient, ties among
    them."""
    sig = np.arange(128, 256) / 128.0
    small = np.concatenate([s * sig * 2.0 ** e for e in range(-6, 1) for s in (1, -1)])  # 1792 values
    rows = []
    for peak in sig:
        x = small[np.abs(small) <= peak]
        x = np.concatenate((x, np.zeros(-x.size % 30)))
        g = np.zeros((x.size // 30, 32))
        g[:, 0], g[:, 2:] = peak, x.reshape(-1, 30)
        rows += [g, np.where(np.arange(32) == 0, -g, g)]
    x = np.concatenate(rows)
    x = np.concatenate((x, np.zeros((-len(x) % 8, 32)))).reshape(1, -1, 1, 256) * 2.0 ** 3
    k, v = (torch.from_numpy(np.ascontiguousarray(x[..., i:i + 128])).cuda().bfloat16() for i in (0, 128))
    c = Cache(1, x.shape[1], 1)
    da.diffattn_kv4_write(k, v, c.t)
    assert np.array_equal(c.entries(), plain.records(x[..., :128], x[..., 128:]))


def test_strided_rows_and_cache():
    """K and V as slices of a fused projection, V1's K as [.., H, 2, 64], a cache with the
    heads outermost, and reads into slices whose surroundings stay as they are."""
    B, N, H, L = 2, 21, 4, 30
    rng = _rng(5)
    fused, fx = _rows(rng, (B, N, 3, H, 128), torch.bfloat16)
    k, v = fused[:, :, 1], fused[:, :, 2]
    a, b = Cache(B, L, H), Cache(B, L, H, head_major=True)
    da.diffattn_kv4_write(k.unflatten(-1, (2, 64)), v, a.t)
    da.diffattn_kv4_write(k, v, b.t)
    want = plain.records(fx[:, :, 1], fx[:, :, 2])
    for c in (a, b):
        assert np.array_equal(c.entries()[:, :N], want) and (c.entries()[:, N:] == SENTINEL).all()
    back = torch.full((B, N, H, 3, 128), 5.0, dtype=torch.float32, device="cuda")
    da.diffattn_kv4_read(b.t, k=back[..., 0, :], v=back[..., 2, :])
    rk, rv = plain.values(want)
    got = back.double().cpu().numpy()
    assert np.array_equal(got[..., 0, :], rk) and np.array_equal(got[..., 2, :], rv)
    assert (got[..., 1, :] == 5.0).all()


def test_positions_and_pages_outside_are_reported():
    B, N, H, L, page = 3, 6, 2, 10, 4
    rng = _rng(6)
    k, kx = _rows(rng, (B, N, H, 128), torch.bfloat16)
    v, vx = _rows(rng, (B, N, H, 128), torch.bfloat16)
    c = Cache(B, L, H, page)
    true = c.table.clone()
    c.table[1, 0], c.table[1, 1] = -1, c.pool
    pos = [7, 0, -2]  # entry 0 runs past the end, entry 1 meets bad pages, entry 2 starts before 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    da.diffattn_kv4_write(k, v, c.t, pos=_i32(pos), dev_status=st, **c.where)
    assert st.item() == -1
    st.zero_()
    kb, vb = da.diffattn_kv4_read(c.t, n_tokens=N, pos=_i32(pos), dtype=torch.float32, dev_status=st, **c.where)
    assert st.item() == -1
    c.table = true
    want = np.full((B, L, H, 144), SENTINEL, np.uint8)
    rec = plain.records(kx, vx)
    want[0, 7:10] = rec[0, :3]
    want[2, 0:4] = rec[2, 2:]
    assert np.array_equal(c.entries(), want)
    rk, rv = plain.values(rec)
    for got, ref in ((kb, rk), (vb, rv)):
        ref = ref.copy()
        ref[0, 3:] = 0
        ref[1] = 0
        ref[2, :2] = 0
        assert np.array_equal(got.double().cpu().numpy(), ref)


def test_inconsistent_offsets_are_skipped():
    H, L = 2, 40
    rng = _rng(7)
    k, kx = _rows(rng, (30, H, 128), torch.bfloat16)
    v, vx = _rows(rng, (30, H, 128), torch.bfloat16)
    c = Cache(4, L, H)
    cu = _i32([0, 10, 8, 20, 31])  # entry 1 decreases, entry 3 ends past the rows
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    da.diffattn_kv4_write(k, v, c.t, cu_seqlens=cu, max_seqlen=12, dev_status=st)
    assert st.item() == -1
    want = np.full((4, L, H, 144), SENTINEL, np.uint8)
    want[0, :10] = plain.records(kx[:10], vx[:10])
    want[2, :12] = plain.records(kx[8:20], vx[8:20])
    assert np.array_equal(c.entries(), want)
    st.zero_()
    kb, vb = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    da.diffattn_kv4_read(c.t, cu_seqlens=cu, max_seqlen=11, k=kb, v=vb, dev_status=st)
    assert st.item() == -1  # entry 2 has 12 rows, more than max_seqlen
    rk, _ = plain.values(want[0, :10])
    assert np.array_equal(kb[:10].double().cpu().numpy(), plain.bf16_round(rk))
    assert (kb[10:] == 3.0).all() and (vb[10:] == 3.0).all()


def test_offsets_past_32_bits():
    """Records more than 2^32 bytes into the pool."""
    H, page = 1, 16
    stride = 5 << 30
    raw = torch.zeros(stride + page * 144, dtype=torch.uint8, device="cuda")
    pool = raw.as_strided((2, page, H, 144), (stride, 144, 144, 1))
    table = _i32([1]).view(1, 1)
    rng = _rng(8)
    k, kx = _rows(rng, (1, page, H, 128), torch.bfloat16)
    v, vx = _rows(rng, (1, page, H, 128), torch.bfloat16)
    da.diffattn_kv4_write(k, v, pool, block_table=table)
    want = plain.records(kx, vx)
    assert np.array_equal(pool[1].cpu().numpy(), want[0]) and not pool[0].any()
    kb, _ = da.diffattn_kv4_read(pool, n_tokens=page, block_table=table, dtype=torch.float32)
    assert np.array_equal(kb.double().cpu().numpy(), plain.values(want)[0])
    q, qx = _rows(rng, (1, 2, 128), torch.bfloat16)
    lam = torch.tensor([0.7], device="cuda")
    out = da.diffattn_fwd_decode_kv4(q, pool, lam, block_table=table)
    ref, bound = plain.decode(qx, want, [0.7], [page], 2)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


# ---- decode ---------------------------------------------------------------------------

def _decode_case(variant, B, Hq, H, L, lens, page=0, seed=0, qscale=1.0, kscale=1.0, vscale=1.0, **extra):
    """Cache, q and lambda of a decode; records past an entry's keys are 0xFF (NaN scales)."""
    rng = _rng(seed)
    kx = plain.bf16_round(rng.standard_normal((B, L, H, 128)) * kscale)
    vx = plain.bf16_round(rng.standard_normal((B, L, H, 128)) * vscale)
    rec = plain.records(kx, vx)
    dirty = rec.copy()
    for b, n in enumerate(lens):
        dirty[b, n:] = 0xFF
    c = Cache(B, L, H, page, seed=seed).set_entries(dirty)
    q, qx = _rows(rng, (B, Hq, 2, 64) if variant == 1 else (B, Hq, 128), torch.bfloat16, qscale)
    lam = rng.uniform(-0.3, 0.95, Hq if variant == 1 else Hq // 2).astype(np.float32)
    return c, rec, q, qx, lam


def _check_decode(variant, c, rec, q, qx, lam, lens, what="", norm=None, **kw):
    li = 0.7778701
    norm = (variant == 1) if norm is None else norm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = da.diffattn_fwd_decode_kv4(
        q, c.t, torch.from_numpy(lam).cuda(), kv_len=_i32(lens), apply_norm=norm,
        lambda_init=torch.full((1,), li, device="cuda") if norm else None, dev_status=st, **c.where, **kw)
    got = out.double().cpu().numpy()
    ref, bound = plain.decode(qx, rec, lam.astype(np.float64), lens, variant, float(np.float32(li)), norm)
    worst = np.max(np.abs(got - ref) / bound) if got.size else 0.0
    assert (np.abs(got - ref) <= bound).all(), f"{what}: {worst:.3f} of the bound"
    assert st.item() == 0
    return out


@pytest.mark.parametrize("Hq,H", [(2, 1), (12, 2), (16, 2), (32, 2), (48, 2), (6, 3)])
@pytest.mark.parametrize("page", [0, 1, 16, 256])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode_v2(Hq, H, page, splits):
    lens = [600, 0, 1, 31, 32, 33, 127, 128, 129, 383]
    case = _decode_case(2, 10, Hq, H, 600, lens, page, seed=Hq + page)
    _check_decode(2, *case, lens, num_splits=splits)


@pytest.mark.parametrize("H", [1, 5])
@pytest.mark.parametrize("page", [0, 4, 64])
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("norm", [True, False])
def test_decode_v1(H, page, splits, norm):
    lens = [500, 0, 1, 64, 129, 447]
    case = _decode_case(1, 6, H, H, 500, lens, page, seed=H + page, qscale=0.5)
    _check_decode(1, *case, lens, num_splits=splits, norm=norm)


@pytest.mark.parametrize("L", [1, 2, 127, 128, 4097, 20000])
def test_decode_lengths(L):
    case = _decode_case(2, 1, 8, 1, L, [L], seed=L)
    _check_decode(2, *case, [L])
    case = _decode_case(1, 1, 2, 2, L, [L], seed=L, qscale=0.125, kscale=0.125, vscale=0.125)
    _check_decode(1, *case, [L])


@pytest.mark.parametrize("qscale,kscale,vscale", [(30.0, 1.0, 1.0), (1e-4, 1e4, 1e4), (1e20, 1e-20, 1e-25),
                                                  (1e-30, 1e30, 1e30), (8.0, 4.0, 1e-3)])
def test_decode_magnitudes(qscale, kscale, vscale):
    lens = [300, 77]
    case = _decode_case(2, 2, 16, 2, 300, lens, seed=9, qscale=qscale, kscale=kscale, vscale=vscale)
    _check_decode(2, *case, lens, num_splits=2)


def test_decode_uneven_value_scales():
    """V rows whose scales differ by 2^40 and rows of zeros, under flat and peaked scores: the
    fp16 products are kept in range by a bound that follows score and scale together."""
    for qs in (0.1, 4.0):
        rng = _rng(10)
        L, H = 400, 2
        kx = plain.bf16_round(rng.standard_normal((1, L, H, 128)))
        size = np.exp2(rng.integers(-20, 21, (1, L, H, 1)).astype(np.float64)) * (rng.random((1, L, H, 1)) > 0.2)
        vx = plain.bf16_round(rng.standard_normal((1, L, H, 128)) * size)
        vx[:, 100:230] = 0.0
        rec = plain.records(kx, vx)
        c = Cache(1, L, H).set_entries(rec)
        q, qx = _rows(rng, (1, 16, 128), torch.bfloat16, qs)
        lam = np.full(8, 0.5, np.float32)
        _check_decode(2, c, rec, q, qx, lam, [L], what=f"q scale {qs}")
        zero = plain.records(kx, np.zeros_like(vx))
        c = Cache(1, L, H).set_entries(zero)
        out = _check_decode(2, c, zero, q, qx, lam, [L])
        assert (out == 0).all()


def test_decode_rising_scores():
    """Scores that rise along the keys: the running maximum is raised chunk after chunk."""
    rng = _rng(11)
    L = 1000
    base = rng.standard_normal(128)
    kx = plain.bf16_round((base * np.linspace(-4, 4, L)[:, None])[None, :, None])
    vx = plain.bf16_round(rng.standard_normal((1, L, 1, 128)))
    rec = plain.records(kx, vx)
    c = Cache(1, L, 1).set_entries(rec)
    qx = plain.bf16_round(np.stack([base, -base] * 4)[None])
    q = torch.from_numpy(qx).cuda().bfloat16()
    _check_decode(2, c, rec, q, qx, np.full(4, 0.6, np.float32), [L], num_splits=1)


def test_decode_equal_large_scores():
    """Keys that are all the same have the same score however large, so every output is the
    plain mean of V: nothing but fp16's rounding of the weights (2^-11 each) and the result's
    (2^-8) is allowed, whichever warps and blocks held the keys."""
    rng = _rng(23)
    L = 1500
    for size in (1.0, 300.0, 1e5):
        kx = plain.bf16_round(np.broadcast_to(rng.standard_normal(128), (1, L, 2, 128)).copy() * size)
        vx = plain.bf16_round(rng.standard_normal((1, L, 2, 128)) + 1.0)
        rec = plain.records(kx, vx)
        held = plain.values(rec)[1]
        qx = plain.bf16_round(np.repeat(kx[0, 0], 8, 0)[None] / size)
        for page, splits in ((0, 0), (0, 1), (0, 5), (2, 3)):
            c = Cache(1, L, 2, page, seed=1).set_entries(rec)
            out = da.diffattn_fwd_decode_kv4(torch.from_numpy(qx).cuda().bfloat16(), c.t, torch.zeros(8, device="cuda"),
                                             num_splits=splits, **c.where).double().cpu().numpy()
            ref = np.repeat(held[0].mean(0), 4, 0)
            allowed = 2.0 ** -10 * np.repeat(np.abs(held[0]).mean(0), 4, 0)
            assert (np.abs(out[0] - ref) <= allowed + 2.0 ** -8 * (np.abs(ref) + allowed)).all(), (size, page, splits)


def test_decode_equal_branches_cancel_exactly():
    case = list(_decode_case(2, 2, 8, 2, 300, [300, 171], seed=12))
    case[2] = case[2].view(2, 4, 2, 128)[:, :, :1].expand(-1, -1, 2, -1).reshape(2, 8, 128).contiguous()
    out = da.diffattn_fwd_decode_kv4(case[2], case[0].t, torch.ones(4, device="cuda"), kv_len=_i32([300, 171]),
                                     num_splits=2)
    assert (out == 0).all()


@pytest.mark.parametrize("L,splits", [(20, 1), (700, 1), (6000, 0)])
def test_decode_flat_scores_and_lambda_near_one(L, splits):
    """Nearly equal branches and lambda near 1, where V1's norm scales up what the difference
    leaves. Branch 1's operand is p_1 - c p_2, so fp16's 2^-11 is allowed on the difference of
    the weights only, and on a tenth of branch 2's for c's own distance from lambda l_1 / l_2
    (scores of standard deviation 0.12 keep l_1 / l_2 within that over any share of the keys);
    fp32 scores and sums take 2^-16 of both, and the result is rounded to bf16."""
    H = 4
    c, rec, q, qx, lam = _decode_case(1, 2, H, H, L, [L, L], seed=L, qscale=0.125, kscale=0.125, vscale=0.125)
    lam = np.array([1.0, 0.97, 1.03, 0.9], np.float32)
    li = np.float32(0.7778701)
    out = da.diffattn_fwd_decode_kv4(q, c.t, torch.from_numpy(lam).cuda(), lambda_init=torch.full((1,), float(li), device="cuda"),
                                     num_splits=splits).double().cpu().numpy()
    for b in range(2):
        for h in range(H):
            k, v = plain.values(rec[b, :, h])
            w = []
            for e in range(2):
                p = np.exp(k[:, 64 * e:64 * e + 64] @ qx[b, h, e] / 8)
                w.append(p / p.sum())
            y = (w[0] - lam[h] * w[1]) @ v
            dy = 2.0 ** -11 * (np.abs(w[0] - lam[h] * w[1]) + 0.1 * lam[h] * w[1]) @ np.abs(v)
            dy += 2.0 ** -16 * (w[0] + lam[h] * w[1]) @ np.abs(v)
            r = np.sqrt((y * y).mean() + 1e-5)
            dy = (dy + np.abs(y) * np.sqrt((dy * dy).mean()) / r) / r * (1 - li)
            y = y / r * (1 - li)
            assert (np.abs(out[b, h] - y) <= dy + 2.0 ** -8 * (np.abs(y) + dy)).all(), (b, h)


def test_decode_nan_stays_where_it_is():
    lens = [200, 200, 200]
    c, rec, q, qx, lam = _decode_case(2, 3, 16, 2, 200, lens, seed=13)
    bad = c.t.clone()
    bad[1, 150, 1, 136:138] = 0xFF  # a NaN V scale of entry 1, head 1
    q = q.clone()
    q[2, 3, 5] = float("nan")  # pair 1 of entry 2
    out = da.diffattn_fwd_decode_kv4(q, bad, torch.from_numpy(lam).cuda(), kv_len=_i32(lens))
    ref, bound = plain.decode(qx, rec, lam.astype(np.float64), lens, 2)
    got = out.double().cpu().numpy()
    nan = np.isnan(got)
    assert nan[1, 4:, :32].all() and nan[2, 1].all()
    clean = np.ones(got.shape, bool)
    clean[1, 4:] = False
    clean[2, 1] = False
    assert (np.abs(got - ref)[clean] <= bound[clean]).all()


def test_decode_bad_page_reads_as_zeros():
    lens = [64, 50]
    c, rec, q, qx, lam = _decode_case(2, 2, 8, 1, 64, lens, page=16, seed=14)
    c.table[0, 1], c.table[1, 2] = -5, 1 << 30
    rec[0, 16:32], rec[1, 32:48] = 0, 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = da.diffattn_fwd_decode_kv4(q, c.t, torch.from_numpy(lam).cuda(), kv_len=_i32(lens), dev_status=st, **c.where)
    assert st.item() == -1
    ref, bound = plain.decode(qx, rec, lam.astype(np.float64), lens, 2)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_decode_lengths_outside_are_clamped():
    c, rec, q, qx, lam = _decode_case(2, 2, 8, 1, 96, [96, 96], seed=15)
    out = da.diffattn_fwd_decode_kv4(q, c.t, torch.from_numpy(lam).cuda(), kv_len=_i32([1 << 30, -7]))
    ref, bound = plain.decode(qx, rec, lam.astype(np.float64), [96, 0], 2)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_decode_strided_and_layouts():
    """q and out as slices; pages of 8 tokens and more give the contiguous cache's result bit
    for bit; smaller pages, and a cache with the heads outermost, go other ways through the
    kernel and stay within the bound."""
    lens = [300, 123]
    c, rec, q, qx, lam = _decode_case(2, 2, 16, 2, 300, lens, seed=16)
    kw = dict(kv_len=_i32(lens), num_splits=3)
    l = torch.from_numpy(lam).cuda()
    base = da.diffattn_fwd_decode_kv4(q, c.t, l, **kw)
    wide = torch.zeros((2, 20, 3, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:18, 1] = q
    out = torch.full((2, 8, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    da.diffattn_fwd_decode_kv4(wide[:, 2:18, 1], c.t, l, out=out[:, :, 0], **kw)
    assert torch.equal(out[:, :, 0], base) and (out[:, :, 1] == 9.0).all()
    for page in (8, 32, 512):
        pc = Cache(2, 300, 2, page, seed=page).set_entries(rec)
        assert torch.equal(da.diffattn_fwd_decode_kv4(q, pc.t, l, **kw, **pc.where), base)
    for other in (Cache(2, 300, 2, 2, seed=2), Cache(2, 300, 2, head_major=True),
                  Cache(2, 300, 2, 16, seed=4, head_major=True)):
        _check_decode(2, other.set_entries(rec), rec, q, qx, lam, lens)
    # a pool whose records are further apart than they are long
    apart = torch.full((2, 300, 2, 160), 0xFF, dtype=torch.uint8, device="cuda")
    apart[..., :144] = c.t
    c.t = apart[..., :144]
    _check_decode(2, c, rec, q, qx, lam, lens)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("page", [0, 2, 8, 128])
def test_decode_ragged_batches(H, page):
    """Many entries of very different lengths: blocks begin and end anywhere in the units."""
    lens = [1, 700, 0, 0, 33, 64, 65, 2, 129, 700, 1, 1, 5, 300, 0]
    case = _decode_case(2, len(lens), 4 * H, H, 700, lens, page, seed=H + page)
    for splits in (0, 1, 2, 7):
        _check_decode(2, *case, lens, num_splits=splits, what=f"splits {splits}")
    lens = [0] * len(lens)
    _check_decode(2, *case, lens)


@pytest.mark.parametrize("Hq,H", [(2, 1), (24, 2), (48, 3), (8, 4), (40, 4)])
@pytest.mark.parametrize("page", [0, 1, 8, 32])
def test_decode_short_caches(Hq, H, page):
    """Entries short enough to stay whole in a block each: no workspace, and empty ones are
    written as zeros; rows and heads around the output stay as they are."""
    lens = [0, 1, 100, 33, 0, 64, 7]
    c, rec, q, qx, lam = _decode_case(2, len(lens), Hq, H, 100, lens, page, seed=Hq + page)
    assert da.diffattn_decode_kv4_workspace_size(*da._binding.decode_kv4_params(q, c.t, None, 0, c.table, 100)) == 0
    wide = torch.full((len(lens), Hq // 2, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    out = _check_decode(2, c, rec, q, qx, lam, lens, out=wide[:, :, 1])
    assert (wide[:, :, 0] == 9.0).all() and (out[0] == 0).all() and (out[4] == 0).all()


def test_two_threads():
    """Two host threads, each on its own stream with its own cache, many calls at once; every
    result equals the same call made alone."""
    import threading
    cases = [_decode_case(2, 2, 16, 2, n, [n, n // 2], seed=n) for n in (2000, 90)]

    def call(i):
        c, rec, q, qx, lam = cases[i]
        da.diffattn_kv4_write(kv[i][0], kv[i][1], c.t, pos=_i32([5, 9]))
        return da.diffattn_fwd_decode_kv4(q, c.t, torch.from_numpy(lam).cuda(), kv_len=_i32([c.L, c.L // 2]))

    kv = [tuple(_rows(_rng(30 + i + j), (2, 1, 2, 128), torch.bfloat16)[0] for j in range(2)) for i in range(2)]
    alone = [call(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs = [call(i) for _ in range(30)]
        s.synchronize()
        wrong.extend(not torch.equal(o, alone[i]) for o in outs)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(wrong) == 60 and not any(wrong)


@pytest.mark.parametrize("variant", [1, 2])
def test_decode_large(variant):
    """The full-size step's cache length and heads at a smaller batch, against 64-bit products
    on the device over a sample of the entries."""
    B, L = 6, 32768
    H, Hq = (16, 16) if variant == 1 else (8, 64)
    g = torch.Generator(device="cuda").manual_seed(17)
    std = 0.125 if variant == 1 else 1.0
    rows = [(torch.randn((B, L, H, 128), generator=g, device="cuda") * std).bfloat16() for _ in range(2)]
    cache = torch.empty((B, L, H, 144), dtype=torch.uint8, device="cuda")
    da.diffattn_kv4_write(rows[0], rows[1], cache)
    lens = [L, L, 1, 20001, L - 1, 0]
    q = (torch.randn((B, Hq, 2, 64) if variant == 1 else (B, Hq, 128), generator=g, device="cuda") * std).bfloat16()
    units = Hq if variant == 1 else Hq // 2
    lam = 0.8 + 0.1 * torch.randn(units, generator=g, device="cuda")
    li = torch.full((1,), 0.7778701, device="cuda")
    out = da.diffattn_fwd_decode_kv4(q, cache, lam, kv_len=_i32(lens), lambda_init=li if variant == 1 else None)
    k, v = da.diffattn_kv4_read(cache, n_tokens=L, dtype=torch.float32)
    for b in (0, 2, 3, 5):
        n = lens[b]
        kd, vd = (t[b, :n].double().transpose(0, 1) for t in (k, v))  # [H, n, 128]
        qd = q[b].double()
        if variant == 1:
            x = torch.einsum("hed,hned->hen", qd, kd.unflatten(-1, (2, 64))) / 8
        else:
            x = torch.einsum("hgd,hnd->hgn", qd.view(H, -1, 128), kd) / 128 ** 0.5
        p = torch.softmax(x, -1)
        o, mag = (torch.einsum("hgn,hnd->hgd", p, t).reshape(-1, 2, 128) for t in (vd, vd.abs()))
        y = o[:, 0] - lam[:, None].double() * o[:, 1]
        # roundings as in kv4_plain.decode, their sum over the keys: p's fp16 rounding (2^-11)
        # and 2^-13 for the scores at these magnitudes, on sum p |v|
        dy = (2.0 ** -11 + 2.0 ** -13) * (mag[:, 0] + lam[:, None].abs() * mag[:, 1])
        if variant == 1:
            r = torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5)
            dy = (dy + y.abs() * torch.sqrt((dy * dy).mean(-1, keepdim=True)) / r) / r * (1 - li)
            y = y / r * (1 - li)
        assert ((out[b].double() - y).abs() <= dy + 2.0 ** -8 * (y.abs() + dy)).all()


def test_decode_is_deterministic_and_default_workspace_agrees():
    lens = [3000, 2047]
    c, rec, q, qx, lam = _decode_case(2, 2, 16, 2, 3000, lens, seed=18)
    l, kl = torch.from_numpy(lam).cuda(), _i32(lens)
    base = da.diffattn_fwd_decode_kv4(q, c.t, l, kv_len=kl)
    n = da.diffattn_decode_kv4_workspace_size(*da._binding.decode_kv4_params(q, c.t, None))
    for fill in (0xFF, 0x00, 0x7F):  # the workspace's contents do not matter
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(da.diffattn_fwd_decode_kv4(q, c.t, l, kv_len=kl, workspace=ws), base)


# ---- together -------------------------------------------------------------------------

def test_serving_run():
    """A prompt through the prefill and into the cache, decode steps that each write their
    token first, and a chunked prefill over what the cache reads back, in a paged cache."""
    B, N, H, Hq, page, steps = 2, 150, 2, 16, 16, 3
    L = 192
    rng = _rng(20)
    c = Cache(B, L, H, page, seed=20)
    lam_np = rng.uniform(0.3, 0.9, Hq // 2).astype(np.float32)
    lam = torch.from_numpy(lam_np).cuda()
    k, kx = _rows(rng, (B, N, H, 128), torch.bfloat16)
    v, vx = _rows(rng, (B, N, H, 128), torch.bfloat16)
    q, _ = _rows(rng, (B, N, Hq, 128), torch.bfloat16)
    da.diffattn_fwd_prefill(q, k, v, lam)
    da.diffattn_kv4_write(k, v, c.t, **c.where)
    rec = plain.records(kx, vx)
    length = _i32([N, N])
    for s in range(steps):
        k1, k1x = _rows(rng, (B, 1, H, 128), torch.bfloat16)
        v1, v1x = _rows(rng, (B, 1, H, 128), torch.bfloat16)
        q1, q1x = _rows(rng, (B, Hq, 128), torch.bfloat16)
        da.diffattn_kv4_write(k1, v1, c.t, pos=length, **c.where)
        length = length + 1
        rec = np.concatenate((rec, plain.records(k1x, v1x)), 1)
        out = da.diffattn_fwd_decode_kv4(q1, c.t, lam, kv_len=length, **c.where)
        n = N + s + 1
        ref, bound = plain.decode(q1x, rec, lam_np.astype(np.float64), [n, n], 2)
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    # the next chunk attends the cached tokens as read back: equal to the prefill over the
    # same values held in a plain tensor
    n, extra = N + steps, 20
    kc, _ = _rows(rng, (B, extra, H, 128), torch.bfloat16)
    vc, _ = _rows(rng, (B, extra, H, 128), torch.bfloat16)
    qc, _ = _rows(rng, (B, extra, Hq, 128), torch.bfloat16)
    kb = torch.empty((B, n + extra, H, 128), dtype=torch.bfloat16, device="cuda")
    vb = torch.empty_like(kb)
    da.diffattn_kv4_read(c.t, k=kb[:, :n], v=vb[:, :n], **c.where)
    kb[:, n:], vb[:, n:] = kc, vc
    got = da.diffattn_fwd_prefill(qc, kb, vb, lam)
    held = [torch.from_numpy(plain.bf16_round(x)).cuda().bfloat16() for x in plain.values(rec)]
    want = da.diffattn_fwd_prefill(qc, torch.cat((held[0], kc), 1), torch.cat((held[1], vc), 1), lam)
    assert torch.equal(got, want)


def test_captured_step_replays_on_another_stream():
    """Write, decode and read captured into one graph on a stream of their own; the replay
    follows the inputs' new contents, and two graphs keep apart."""
    B, H, Hq, L = 3, 2, 16, 300
    rng = _rng(21)
    c, rec, q, qx, lam = _decode_case(2, B, Hq, H, L, [L] * B, seed=21)
    l, length, pos = torch.from_numpy(lam).cuda(), _i32([101, 300, 1]), _i32([100, 299, 0])
    k, _ = _rows(rng, (B, 1, H, 128), torch.bfloat16)
    v, _ = _rows(rng, (B, 1, H, 128), torch.bfloat16)
    s = torch.cuda.Stream()

    def step():
        da.diffattn_kv4_write(k, v, c.t, pos=pos)
        return da.diffattn_fwd_decode_kv4(q, c.t, l, kv_len=length), *da.diffattn_kv4_read(c.t, n_tokens=1, pos=pos)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = step()
        graphs.append((graph, outs))
    for seed in (1, 2):
        r = _rng(100 + seed)
        k.copy_(_rows(r, k.shape, torch.bfloat16)[0])
        v.copy_(_rows(r, v.shape, torch.bfloat16)[0])
        q.copy_(_rows(r, q.shape, torch.bfloat16)[0])
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for graph, outs in graphs:
            for t in outs:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_stream_argument():
    """Work given a stream runs there, and what the call allocates belongs to that stream."""
    lens = [2000]
    c, rec, q, qx, lam = _decode_case(2, 1, 16, 2, 2000, lens, seed=22)
    l = torch.from_numpy(lam).cuda()
    want = da.diffattn_fwd_decode_kv4(q, c.t, l)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(8):
        outs.append(da.diffattn_fwd_decode_kv4(q, c.t, l, stream=s))
        torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")  # the current stream's allocations
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
