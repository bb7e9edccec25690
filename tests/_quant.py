"""Plain 64-bit forms of the 8-bit cache and of the attentions over it, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

E_MIN = -110


def quantise(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """float64 rows [..., D] -> (the value of each e4m3 code, exponent byte): the smallest
    e >= -110 with max|x| <= 448 2^e; x 2^-e to the nearest e4m3, ties to even, at e = 120 at most
    240 (no more fits bf16); a row with a
    non-finite value is (NaN, 255)."""
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    a = np.abs(x).max(-1)
    e = np.full(a.shape, E_MIN)
    while (over := a > 448.0 * 2.0**e).any():
        e = e + over
    y = x * 2.0 ** -e[..., None].astype(np.float64)
    # e4m3: 3 fraction bits, exponents from -6; below, steps of 2^-9
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0**-30))), -6) - 3)
    code = np.rint(y / step) * step  # rint: ties to even
    code = np.where((e == 120)[..., None], np.clip(code, -240, 240), code)  # 256 * 2^120 is no bf16 number
    return np.where(bad[..., None], np.nan, code), np.where(bad, 255, e + 127).astype(np.uint8)


def code_values(c: torch.Tensor) -> np.ndarray:
    """The values of a float8_e4m3fn tensor as float64."""
    b = c.view(torch.uint8).cpu().numpy().astype(np.int64)
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0**-9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def widen(code: torch.Tensor, ebyte: torch.Tensor) -> np.ndarray:
    """float64 values of codes [B, L, H, D] with exponent bytes [B, H, S]."""
    e = ebyte[:, :, : code.shape[1]].cpu().numpy().astype(np.float64).transpose(0, 2, 1)[..., None]
    return code_values(code) * np.where(e == 255, np.nan, 2.0 ** (e - 127))


def attention(q, k, v, scale):
    """float64 softmax(scale q k^T) v of one sequence, q [R, Hq, D], k, v [n, Hkv, D], and the bound
    of the kernel's error: every weight is rounded to bf16 (2^-8 of it) and so is the result
    (2^-8 of it, and |result| <= A = sum_j p_j |v_j|), so 2^-7 A, and 2^-10 A for the second order,
    the approximate exponential (2^-22) and the sums; the scores' fp32 products add
    delta = D 2^-23 max_j scale sum_d |q_d k_jd| to an exponent, 2 delta A to the result (through the
    weight and through the sum)."""
    R, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, tol = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    if k.shape[0] == 0:
        return out, tol
    for h in range(Hq):
        kk, vv = k[:, h // g], v[:, h // g]
        z = scale * (q[:, h] @ kk.T)
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        delta = D * 2.0**-23 * scale * (np.abs(q[:, h]) @ np.abs(kk).T).max(1, keepdims=True)
        out[:, h] = p @ vv
        tol[:, h] = (2.0**-7 + 2.0**-10 + 2 * delta) * (p @ np.abs(vv)) + 1e-30
    return out, tol


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def random_cache(rng, B, L, Hkv, D, spread=1.0):
    """Codes and exponent bytes of rows whose magnitude differs by position: (k, v, k_exp, v_exp) on the CPU."""
    S = -(-L // 16) * 16
    out = []
    for _ in range(2):
        x = rng.standard_normal((B, L, Hkv, D)) * 2.0 ** (spread * rng.standard_normal((B, L, Hkv, 1)))
        c, e = quantise(f64(bf16(x)))
        eb = np.full((B, Hkv, S), 0xAB, np.uint8)  # the padding is never used
        eb[:, :, :L] = e.transpose(0, 2, 1)
        out.append((torch.from_numpy(c).float().to(torch.float8_e4m3fn), torch.from_numpy(eb)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def default_scale(D):
    return 1.0 / math.sqrt(D)
