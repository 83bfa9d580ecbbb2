"""Grouped products of plain operands, 8-bit-integer row quantisation and the AdamW step, in float64.

Definitions: W_g is rows gN .. gN + N of w; expert g's rows are offs[g] .. offs[g + 1].
"""
from __future__ import annotations

import numpy as np

from .codecs import bf16_bits_to_f64, e4m3_decode, e4m3_encode

TINY = 2.0 ** -126
TOP = 1.875


def _experts(offs):
    return [(g, slice(int(offs[g]), int(offs[g + 1]))) for g in range(len(offs) - 1)]


def dense_gemm_fwd(x, w, offs, N):
    """(Y [M, N], sum |x w|) of bf16 bit patterns x [M, K], w [G*N, K]."""
    x, w = bf16_bits_to_f64(x), bf16_bits_to_f64(w)
    out = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N))
    for g, r in _experts(offs):
        wg = w[g * N:(g + 1) * N]
        out[0][r], out[1][r] = x[r] @ wg.T, np.abs(x[r]) @ np.abs(wg).T
    return out


def dense_gemm_dgrad(dy, w, offs, N, K):
    """(dX [M, K], sum |dy w|)."""
    dy, w = bf16_bits_to_f64(dy), bf16_bits_to_f64(w)
    out = np.zeros((dy.shape[0], K)), np.zeros((dy.shape[0], K))
    for g, r in _experts(offs):
        wg = w[g * N:(g + 1) * N]
        out[0][r], out[1][r] = dy[r] @ wg, np.abs(dy[r]) @ np.abs(wg)
    return out


def dense_gemm_wgrad(dy, x, offs):
    """(dW [G, N, K], sum |dy x|)."""
    dy, x = bf16_bits_to_f64(dy), bf16_bits_to_f64(x)
    shape = (len(offs) - 1, dy.shape[1], x.shape[1])
    out = np.zeros(shape), np.zeros(shape)
    for g, r in _experts(offs):
        out[0][g], out[1][g] = dy[r].T @ x[r], np.abs(dy[r]).T @ np.abs(x[r])
    return out


def int8_quantize_rows(v):
    """(codes int8, scales float32) of float64 rows: s = fl32(amax / 127), q = nearest even of 127 v / amax."""
    v = np.asarray(v, np.float64)
    amax = np.abs(v).max(axis=1)
    safe = np.where(amax > 0, amax, 1.0)
    q = np.rint(127.0 * v / safe[:, None]).astype(np.int8)
    return q, np.where(amax > 0, amax / 127.0, 1.0).astype(np.float32)


def int8_gemm_fwd(qx, sx, qw, sw, offs, N):
    """Y [M, N] float64; the integer sums are exact."""
    y = np.zeros((qx.shape[0], N))
    for g, r in _experts(offs):
        acc = qx[r].astype(np.float64) @ qw[g * N:(g + 1) * N].astype(np.float64).T
        y[r] = acc * sx[r].astype(np.float64)[:, None] * sw[g * N:(g + 1) * N].astype(np.float64)[None]
    return y


def _block_max(v):
    pad = np.zeros(-(-v.size // 128) * 128)
    pad[:v.size] = np.abs(v)
    return pad.reshape(-1, 128).max(axis=1)


def _spread(s, n):
    return np.repeat(s.astype(np.float64), 128)[:n]


def adamw_pack_m(m):
    """E4M3 codes and float32 scales per 128 of a float64 first moment."""
    s = np.maximum(_block_max(m) / 448.0, TINY).astype(np.float32)
    return e4m3_encode(np.clip(m / _spread(s, m.size), -448, 448)), s


def adamw_unpack_m(q, s):
    return e4m3_decode(q) * _spread(s, q.size)


def adamw_v_values():
    """The 256 values of the second moment's code: 0, then (1 + f / 8) 2^(E - 31) of code 8 E + f."""
    c = np.arange(256)
    return np.where(c > 0, (1 + (c % 8) / 8.0) * 2.0 ** (c // 8 - 31.0), 0.0)


def adamw_pack_v(v):
    """Codes and float32 scales of a float64 second moment: nearest value, ties to the even code, a value
    that is not zero at least code 1."""
    s = np.maximum(_block_max(v) / TOP, TINY).astype(np.float32)
    y = v / _spread(s, v.size)
    table = adamw_v_values()
    hi = np.clip(np.searchsorted(table, y), 1, 255)
    lo = hi - 1
    up, down = table[hi] - y, y - table[lo]
    q = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(v > 0, np.maximum(q, 1), 0).astype(np.uint8), s


def adamw_unpack_v(q, s):
    return adamw_v_values()[q] * _spread(s, q.size)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, wd, scale=1.0):
    """One step in float64: (p, m, v)."""
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(v / (1 - beta2 ** step)) + eps
    return p * (1 - lr * wd) - lr * (m / (1 - beta1 ** step)) / root, m, v
