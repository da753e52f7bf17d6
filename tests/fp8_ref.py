"""The 8-bit operators' definitions in 64 bits on the CPU (numpy), for their
tests: e4m3 values by enumeration, scales by one fp32 division, products of
the values the codes stand for."""
import numpy as np
import torch

FLOOR = np.float32(2.0 ** -100)
_E = np.arange(128) // 8
_F = np.arange(128) % 8
VALUES = np.where(_E == 0, _F * 2.0 ** -9, (8 + _F) * 2.0 ** (_E.astype(np.float64) - 10))[:127]   # 127: NaN


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def values_of(q: torch.Tensor) -> np.ndarray:
    """The values of e4m3 codes."""
    b = q.detach().cpu().view(torch.uint8).numpy()
    v = np.append(VALUES, np.nan)[b & 127]
    return np.where(b & 128, -v, v)


def nearest_code(v: np.ndarray) -> np.ndarray:
    """Code of the nearest e4m3 value of finite v (|v| < 464), ties to even."""
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    a = np.abs(v)
    lo, hi = np.searchsorted(mid, a), np.searchsorted(mid, a, side="right")
    c = np.where(lo == hi, lo, lo + lo % 2)
    return (c | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale(amax: np.ndarray) -> np.ndarray:
    return np.maximum(amax.astype(np.float32), FLOOR) / np.float32(448)


def quantize_rows(x: torch.Tensor):
    """(codes uint8 [M,K], scales fp32 [ceil(K/128), M])"""
    v = f64(x)
    M, K = v.shape
    kb = -(-K // 128)
    codes, s = np.zeros((M, K), np.uint8), np.zeros((kb, M), np.float32)
    for b in range(kb):
        part = v[:, b * 128:(b + 1) * 128]
        s[b] = scale(np.abs(part).max(axis=1))
        codes[:, b * 128:(b + 1) * 128] = nearest_code(part / s[b].astype(np.float64)[:, None])
    return codes, s


def quantize_tiles(w: torch.Tensor):
    """(codes uint8 [N,K], scales fp32 [ceil(N/128), ceil(K/128)])"""
    v = f64(w)
    N, K = v.shape
    codes, s = np.zeros((N, K), np.uint8), np.zeros((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            s[i, j] = scale(np.abs(v[at]).max(keepdims=True)[0])[0]
            codes[at] = nearest_code(v[at] / np.float64(s[i, j]))
    return codes, s


def spread(s: np.ndarray, R: int, C: int) -> np.ndarray:
    return np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:R], 128, 1)[:, :C]


def rows_value(codes: np.ndarray, s: np.ndarray) -> np.ndarray:
    return values_of(torch.from_numpy(codes)) * np.repeat(s.astype(np.float64).T, 128, 1)[:, :codes.shape[1]]


def tiles_value(codes: np.ndarray, s: np.ndarray) -> np.ndarray:
    return values_of(torch.from_numpy(codes)) * spread(s, *codes.shape)


def half_step(dt: torch.dtype) -> float:
    """Rounding to dt is off by at most this share of the value."""
    return torch.finfo(dt).eps / 2


def product_bound(exact: np.ndarray, mass: np.ndarray, terms: int, dt: torch.dtype) -> np.ndarray:
    """How far one rounding to dt of an fp32 sum of `terms` terms of absolute
    sum `mass` may be from `exact`: each addition (and the scales' product) off
    by at most 2^-24 of the running sum, MFMA's by at most 2^-23 of it."""
    acc = 2.0 ** -23 * (terms + 4) * mass
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0   # half of fp16's smallest step
    return half_step(dt) * (np.abs(exact) + acc) + acc + tiny
