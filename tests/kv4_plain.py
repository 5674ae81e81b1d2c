"""Plain 64-bit forms of the 4-bit KV cache operators, for the tests: quantising rows into
records, the values of records, and differential decode attention over them with a bound on
what the kernel's roundings can add up to."""
from __future__ import annotations

import numpy as np
import torch

RECORD = 144
GROUP = 32


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float64/float32 values rounded to bf16 (nearest, ties to even), as float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()
    return t.double().numpy()


def bf16_bits(x: np.ndarray) -> np.ndarray:
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()
    return t.view(torch.int16).numpy().view(np.uint16)


def quantise(rows: np.ndarray):
    """Rows [..., 128] (bf16 values) -> code bytes [..., 64], scales [..., 4] (float64)."""
    x = np.asarray(rows, dtype=np.float64).reshape(*rows.shape[:-1], 4, GROUP)
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[..., None], x, 0.0)
    size = np.abs(x).max(-1)
    peak = np.where((x == -size[..., None]).any(-1), -size, size)
    zero = size < 2.0 ** -100
    scale = np.where(zero, 0.0, peak / -8.0)
    n = np.clip(np.rint(x / np.where(zero, 1.0, scale)[..., None]), -8, 7)
    n = np.where((zero | ~finite)[..., None], 0, n).astype(np.int64) + 8
    scale = np.where(finite, scale, np.nan)
    n = n.reshape(*rows.shape).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale


def records(k: np.ndarray, v: np.ndarray) -> np.ndarray:
    (ck, sk), (cv, sv) = quantise(k), quantise(v)

    def scale_bytes(s):
        bits = bf16_bits(np.nan_to_num(s, nan=0.0))
        bits = np.where(np.isnan(s), np.uint16(0x7FC0), bits).astype("<u2")
        return np.ascontiguousarray(bits).view(np.uint8)
    return np.concatenate((ck, cv, scale_bytes(sk), scale_bytes(sv)), -1)


def values(rec: np.ndarray):
    """Records [..., 144] -> K, V rows [..., 128] in float64."""
    def rows(codes, sb):
        n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 128).astype(np.float64) - 8
        bits = np.ascontiguousarray(sb).view("<u2").astype(np.uint32) << 16
        return n * np.repeat(bits.view(np.float32).astype(np.float64), GROUP, -1)
    return rows(rec[..., :64], rec[..., 128:136]), rows(rec[..., 64:128], rec[..., 136:144])


def decode(q, rec, lam, kv_len, variant, lambda_init=None, apply_norm=False, eps=1e-5):
    """q [B, Hq, 128] or [B, H, 2, 64], rec [B, L, H, 144] -> (out [B, units, 128], bound).

    The bound, element by element. A probability times a V scale is rounded to fp16 (2^-11; the
    kernel's p_1 - c p_2 for branch 1 has 0 <= c p_2 <= 1.25 p_1, and 2^-11 of its size for branch
    1 and 2^-11 |c / l_1 - lambda / l_2| p_2 for branch 2 add up to no more than with c = 0 unless
    a key has c p_2 > p_1 and c is over 5 lambda l_1 / l_2, and then to 1.5 times that at most);
    fp32 rounding of the scores moves x by at most 40 steps of 2^-24 on the sum of magnitudes
    sum |q| |scale| 24 (nibbles to 15 and the start of 8, products added in MMAs of 16 and then
    over 4 groups), and p by that times ln 2 in relative terms, numerator and denominator
    alike; the log2-domain factors, ex2 (2^-22), the sums and the joins take 2^-18. All of it
    is relative to sum p |v| / sum p of a branch. A product that fp16 holds as a subnormal is
    off by up to 2^-25 instead, where the largest probability times the largest V scale is at
    least 2^8, and a code is at most 8. The result is rounded to bf16 (2^-8). With
    the norm, dy moves y / rms(y) by at most (|dy| + |y| rms(dy) / rms(y)) / rms(y)."""
    q = np.asarray(q, dtype=np.float64)
    B, H = q.shape[0], rec.shape[2]
    units = q.shape[1] if variant == 1 else q.shape[1] // 2
    out, bound = np.zeros((B, units, 128)), np.zeros((B, units, 128))
    for b in range(B):
        n = int(kv_len[b])
        for u in range(units):
            ys, errs = [], []
            for e in range(2):
                if variant == 1:
                    h, d = u, 64
                    qv = np.zeros(128)
                    qv[64 * e:64 * e + 64] = q[b, u, e]
                else:
                    h, d, qv = (2 * u + e) // (q.shape[1] // H), 128, q[b, 2 * u + e]
                if n == 0:
                    ys.append(np.zeros(128))
                    errs.append(np.zeros(128))
                    continue
                k, v = values(rec[b, :n, h])
                x = k @ qv / np.sqrt(d)
                p = np.exp(x - x.max()) if np.isfinite(x).all() else np.full(n, np.nan)
                p = p / p.sum()
                scales = np.ascontiguousarray(rec[b, :n, h, 128:136]).view("<u2").astype(np.uint32) << 16
                scales = np.abs(scales.view(np.float32).astype(np.float64))
                moved = (scales @ np.abs(qv).reshape(4, GROUP).sum(-1)) * 24 / np.sqrt(d) * 40 * 2.0 ** -24
                rel = 2.0 ** -11 + 2 * np.max(moved) + 2.0 ** -18
                ys.append(p @ v)
                vs = np.ascontiguousarray(rec[b, :n, h, 136:144]).view("<u2").astype(np.uint32) << 16
                vs = np.abs(vs.view(np.float32).astype(np.float64)).max()
                errs.append(rel * (p @ np.abs(v)) + n * 8 * 2.0 ** -33 * p.max() * vs)
            y = ys[0] - lam[u] * ys[1]
            dy = errs[0] + abs(lam[u]) * errs[1] + 1e-30
            if apply_norm:
                r = np.sqrt((y * y).mean() + eps)
                dy = (dy + np.abs(y) * np.sqrt((dy * dy).mean()) / r) / r * (1 - lambda_init)
                y = y / r * (1 - lambda_init)
            out[b, u] = y
            bound[b, u] = dy + 2.0 ** -8 * (np.abs(y) + dy)
    return out, bound
