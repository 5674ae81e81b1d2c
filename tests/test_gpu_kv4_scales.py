"""The decode over a 4-bit cache whose V rows differ in size from key to key: the softmax's sums
follow the scores alone, whatever the V scales. Against plain 64-bit attention over the cache's
values, within kv4_plain.decode's bound."""
import numpy as np
import pytest
import torch

import differential_attention_05_b200 as da

import kv4_plain as plain
from test_gpu_kv4 import Cache, _check_decode, _rng, _rows

pytestmark = pytest.mark.gpu


def _sized(variant, H, size, seed, qscale=0.5):
    """A cache of one entry with normal rows, V's times `size` [n], q and lambda."""
    rng = _rng(seed)
    n = size.size
    kx = plain.bf16_round(rng.standard_normal((1, n, H, 128)))
    vx = plain.bf16_round((rng.standard_normal((1, n, H, 128)) + 1.0) * size[None, :, None, None])
    rec = plain.records(kx, vx)
    q, qx = _rows(rng, (1, H, 2, 64) if variant == 1 else (1, 8 * H, 128), torch.bfloat16, qscale)
    lam = rng.uniform(-0.3, 0.95, H if variant == 1 else 4 * H).astype(np.float32)
    return Cache(1, n, H).set_entries(rec), rec, q, qx, lam


@pytest.mark.parametrize("H", [1, 2, 4, 8])
@pytest.mark.parametrize("power", [20, 36, 60, 90])
def test_keys_of_zero_value_count(H, power):
    """Half the keys have V = 0 and half V of 2^power, all with the same score, and the output is
    half of it: the zeros first and last, and in turn by 32 (the keys of a warp's chunk) and by
    blocks' shares."""
    n = 1024
    for run in (32, 64, 128, n // 2):
        for first in (0, 1):
            size = np.where((np.arange(n) // run + first) % 2, 2.0 ** power, 0.0)
            case = _sized(2, H, size, run, qscale=0.0)
            for splits in (1, 2, 4, 0):
                out = _check_decode(2, *case, [n], num_splits=splits, what=f"{run} {first} {splits}")
                assert torch.isfinite(out).all()


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("H", [1, 2, 4])
def test_sizes_along_the_keys(variant, H):
    """V rows that grow or shrink along the keys, over 2^40 to the whole range of the type."""
    n = 640
    for lo, hi in ((-20, 20), (-99, -50), (-99, 120), (60, 120)):
        for size in (np.linspace(lo, hi, n), np.linspace(hi, lo, n), np.where(np.arange(n) < n // 2, lo, hi)):
            # V1's norm squares the output in fp32, which holds sizes to 2^60 or so
            norm = variant == 1 and abs(lo) < 40 and abs(hi) < 40
            case = _sized(variant, H, np.exp2(size), 7)
            for splits in (1, 3, 0):
                _check_decode(variant, *case, [n], norm=norm, num_splits=splits, what=f"{lo} {hi} {splits}")


@pytest.mark.parametrize("power", [-99, -88, 100, 120])
def test_small_probabilities_at_the_ends_of_the_range(power):
    """Scores over 20 powers of two with V at the smallest and the largest sizes: what lies far
    below the largest probability still adds up."""
    n = 2048
    case = list(_sized(2, 4, np.full(n, 2.0 ** power), 8))
    y = np.full(n, -14.0)
    y[5] = 0.0
    kx = np.repeat(np.repeat(y[None, :, None, None], 4, 2), 128, 3)
    rec = case[1]
    vx = plain.values(rec)[1]
    vx[:, 5] = -vx[:, 5].mean(0)  # one key against many
    case[1] = rec = plain.records(plain.bf16_round(kx), plain.bf16_round(vx))
    case[0] = Cache(1, n, 4).set_entries(rec)
    qx = np.full((1, 32, 128), np.sqrt(128) / 128 / np.log2(np.e))
    case[3] = plain.bf16_round(qx)
    case[2] = torch.from_numpy(case[3]).cuda().bfloat16()
    for splits in (1, 4, 0):
        _check_decode(2, *case, [n], num_splits=splits)


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("H", [1, 2, 4, 8])
def test_a_nan_stays_in_its_group_of_channels(variant, H):
    """Rows with a NaN or an infinity, as the write holds them: their groups of 32 channels come
    out as NaN for every query of the head, all other channels as without them."""
    n, B = 600, 3
    rng = _rng(50 + H)
    k, v = (plain.bf16_round(rng.standard_normal((B, n, H, 128))) for _ in range(2))
    lost = np.zeros((B, H, 4), bool)
    for b, t, h, c, x in ((0, 0, 0, 5, np.nan), (0, 470, 0, 40, np.inf), (1, 301, H - 1, 127, -np.inf),
                          (1, 302, H - 1, 127, np.nan), (2, 599, H // 2, 70, np.nan), (2, 40, H // 2, 0, np.inf)):
        v[b, t, h, c] = x
        lost[b, h, c // 32] = True
    rec = plain.records(k, v)
    c = Cache(B, n, H)
    t = [torch.from_numpy(x).cuda().bfloat16() for x in (k, v)]
    da.diffattn_kv4_write(*t, c.t)
    assert np.array_equal(c.entries(), rec)
    q, qx = _rows(rng, (B, H, 2, 64) if variant == 1 else (B, 8 * H, 128), torch.bfloat16, 0.5)
    units = H if variant == 1 else 4 * H
    lam = rng.uniform(0.3, 0.95, units).astype(np.float32)
    ref, bound = plain.decode(qx, plain.records(k, np.where(np.isfinite(v), v, 0.0)), lam.astype(np.float64), [n] * B, variant)
    # the channels that are compared are the other groups', whose codes are the same in both
    gone = np.repeat(np.repeat(lost, units // H, 1), 32, 2)
    kv_len = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for splits in (0, 1, 4):
        out = da.diffattn_fwd_decode_kv4(q, c.t, torch.from_numpy(lam).cuda(), kv_len=kv_len, apply_norm=False,
                                         num_splits=splits).double().cpu().numpy()
        assert np.isnan(out[gone]).all()
        assert (np.abs(out - ref)[~gone] <= bound[~gone]).all(), splits


def test_products_far_below_the_largest():
    """One key has the largest probability and the largest V scale, just over a power of two, but
    the value 0 outside channels 0, 32, 64 and 96; all others have products of 2^-29 to 2^-33 of
    that, every key of an entry the same, so that their fp16 roundings add up: still no more than
    2^-25 each where the largest product is 2^8."""
    B, n, H = 48, 512, 4
    y = np.linspace(-24.0, -28.0, B)
    kx = np.repeat(np.repeat(np.repeat(y[:, None, None, None], n, 1), H, 2), 128, 3)
    vx = np.full((B, n, H, 128), 2.0 ** -5)
    kx[:, 7], vx[:, 7] = 0.0, 0.0
    vx[:, 7, :, ::32] = 8.0625
    vx[:, :7, :, 1::2] *= -1.0
    rec = plain.records(plain.bf16_round(kx), plain.bf16_round(vx))
    qx = plain.bf16_round(np.full((B, 2 * H, 128), np.sqrt(128) / 128 / np.log2(np.e)))
    lam = np.zeros(H, np.float32)
    q = torch.from_numpy(qx).cuda().bfloat16()
    for splits in (1, 0):
        _check_decode(2, Cache(B, n, H).set_entries(rec), rec, q, qx, lam, [n] * B, num_splits=splits)


@pytest.mark.parametrize("channel,power", [(32, -31), (33, -27), (62, -30), (95, -26)])
def test_small_elements_of_q_that_count(channel, power):
    """A row of q whose largest element meets small keys, while one at the least size that is
    held exactly in its channel decides the scores, over keys as much larger."""
    n, H = 700, 2
    rng = _rng(70)
    for size in (1.0, 1.9921875):  # all bits of the significand
        qx = np.zeros((1, 4 * H, 128))
        qx[..., 0] = 1.0
        qx[..., channel] = size * 2.0 ** power
        kx = rng.standard_normal((1, n, H, 128)) * 2.0 ** -20
        at = channel // 32 * 32
        kx[..., at:at + 32] = rng.uniform(-30, 30, (1, n, H, 32)) * 2.0 ** -power
        vx = rng.standard_normal((1, n, H, 128))
        rec = plain.records(plain.bf16_round(kx), plain.bf16_round(vx))
        q = torch.from_numpy(qx).cuda().bfloat16()
        _check_decode(2, Cache(1, n, H).set_entries(rec), rec, q, qx, np.full(2 * H, 0.5, np.float32), [n])
