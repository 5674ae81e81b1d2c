"""The decode over a 4-bit cache where its two branches attend different keys: scores set key by
key, against plain 64-bit attention over the cache's values.

The bound is kv4_plain.decode's. Branch 1's operand is p_1 - c p_2 with 0 <= c p_2 <= 1.25 p_1 for
every key; its fp16 rounding moves O_1 by at most 2^-11 |p_1 - c p_2| |v|, branch 2's moves
O_1 / l_1 - lambda O_2 / l_2 by 2^-11 p_2 |v| times |c / l_1 - lambda / l_2|. Where c p_2 <= p_1, both
make at most 2^-11 (p_1 / l_1 + |lambda| p_2 / l_2) |v|, the bound's first term, whatever c is; they
do so too where c p_2 is between that and 1.25 p_1, unless c is over 5 lambda l_1 / l_2. The scores
here have no key or next to none of that kind: a branch 2 that rises does so by more than the
log2(1.25) in between."""
import numpy as np
import pytest
import torch

import differential_attention_05_b200 as da

import kv4_plain as plain
from test_gpu_kv4 import Cache, _check_decode, _rng

pytestmark = pytest.mark.gpu


def _scored(variant, y, H, seed, vx=None):
    """A cache of one entry whose keys have the log2 scores y [2, n] for the branches of every
    head's first unit, and the branches exchanged for the second (V1: for every other head).
    Channels 0..31 of K hold branch 1's scores and 64..95 branch 2's, each channel the same, so
    the codes are exact; the other channels meet zeros of q."""
    rng = _rng(seed)
    n = y.shape[1]
    kx = rng.standard_normal((1, n, H, 128))
    for e in range(2):
        kx[..., 64 * e:64 * e + 32] = y[e][None, :, None, None]
    if vx is None:
        vx = rng.uniform(-1, 1, (1, n, H, 128))
    rec = plain.records(plain.bf16_round(kx), plain.bf16_round(vx))
    size = np.sqrt(64 if variant == 1 else 128) / (32 * np.log2(np.e))
    if variant == 1:
        qx = np.zeros((1, H, 2, 64))
        qx[..., :32] = size
        for h in range(1, H, 2):  # K_1 and K_2 exchanged
            rec[:, :, h] = plain.records(*(plain.bf16_round(x[:, :, h]) for x in (np.roll(kx, 64, -1), vx)))
        units = H
    else:
        qx = np.zeros((1, H, 2, 2, 128))  # [., heads, pairs, branches, .]
        for pair in range(2):
            for e in range(2):
                at = 64 * (e ^ pair)
                qx[:, :, pair, e, at:at + 32] = size
        qx = qx.reshape(1, 4 * H, 128)
        units = 2 * H
    qx = plain.bf16_round(qx)
    lam = np.resize(np.array([0.8, 0.8, 1.0, 0.95, 0.3, -0.4, 0.6, 1.2], np.float32), units)
    return Cache(1, n, H).set_entries(rec), rec, torch.from_numpy(qx).cuda().bfloat16(), qx, lam


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("H", [1, 2, 4, 8])
def test_branch_2_rises_behind_a_shared_sink(variant, H):
    """Eight keys that both branches attend, a background far below, and further on 96 keys that
    branch 2 attends more than the sink, beginning at chunks of every residue modulo 4."""
    warps = 4 if H == 1 else (2 if H == 2 else 1)  # of a head: a chunk is 32 keys of each
    for low in (-12.0, -30.0):
        for top in (4.0, 5.9):
            for begin in (2, 4, 5, 6, 7, 13):
                y = np.full((2, 17 * 32 * warps), low)
                y[:, :8] = 0.0
                y[1, begin * 32 * warps:begin * 32 * warps + 96 * warps] = top
                case = _scored(variant, y, H, begin)
                for splits in (1, 0):
                    _check_decode(variant, *case, [y.shape[1]], num_splits=splits, what=f"{low} {top} {begin} {splits}")


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("H", [1, 4])
def test_single_keys_above_a_shared_sink(variant, H):
    """Scattered scores, a sink at key 0 of both branches, and one to three later keys of branch 2
    that lie above it."""
    rng = _rng(40)
    for sink in (10.0, 14.0):
        for above in (3.0, 5.8):
            for chunks in ((3,), (5,), (6,), (7,), (13,), (5, 6, 13)):
                y = rng.standard_normal((2, 16 * 32))
                y[:, 0] = sink
                y[1, [32 * i + 11 for i in chunks]] = sink + above
                case = _scored(variant, y, H, 41)
                for splits in (1, 0):
                    _check_decode(variant, *case, [y.shape[1]], num_splits=splits, what=f"{sink} {above} {chunks}")


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("H", [1, 4])
@pytest.mark.parametrize("slope", [0.02, 0.05, 0.13, 0.6])
def test_branches_along_opposite_slopes(variant, H, slope):
    """One branch's scores fall along the keys, the other's rise, in units of both orders."""
    n = 1024
    y = np.array([[-1.0], [1.0]]) * slope * np.minimum(np.arange(n), 60 / slope)
    case = _scored(variant, y, H, 42)
    for splits in (1, 0):
        _check_decode(variant, *case, [n], num_splits=splits)


@pytest.mark.parametrize("variant", [1, 2])
def test_branches_on_keys_of_their_own(variant):
    """Half the keys are branch 1's, half branch 2's, in runs of 32 to 256 keys, with either
    branch's first, over several entries that share blocks."""
    for run in (32, 96, 256):
        for first in (0, 1):
            n = 1536
            own = (np.arange(n) // run + first) % 2
            y = np.stack((np.where(own == 0, 6.0, -6.0), np.where(own == 1, 6.0, -6.0)))
            case = _scored(variant, y, 4, run)
            for splits in (1, 5):
                _check_decode(variant, *case, [n], num_splits=splits, what=f"{run} {first} {splits}")


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("L", [40, 3000])
def test_empty_entries_are_zero_whatever_lambda_and_eps(variant, L):
    """No key gives a zero row: with norm_eps = 0, which the norm would divide by, and a lambda
    that is no number; in caches short enough to stay whole and in ones that are shared."""
    B, H = 3, 2
    rng = _rng(60)
    rec = plain.records(*(plain.bf16_round(rng.standard_normal((B, L, H, 128))) for _ in range(2)))
    c = Cache(B, L, H).set_entries(rec)
    units = H if variant == 1 else 4 * H
    q = torch.randn((B, H, 2, 64) if variant == 1 else (B, 8 * H, 128), device="cuda").bfloat16()
    lam = torch.full((units,), 0.5, device="cuda")
    lam[1] = float("nan")
    kv_len = torch.tensor([0, L, 0], dtype=torch.int32, device="cuda")
    li = torch.full((1,), 0.2, device="cuda") if variant == 1 else None
    for splits in (0, 1, 3):
        for lens in (kv_len, torch.zeros_like(kv_len)):
            out = da.diffattn_fwd_decode_kv4(q, c.t, lam, kv_len=lens, lambda_init=li, norm_eps=0.0, num_splits=splits)
            empty = lens == 0
            assert (out[empty] == 0).all(), splits
            assert torch.isfinite(out[~empty][:, [0]]).all() and out[~empty][:, 1].isnan().all()
