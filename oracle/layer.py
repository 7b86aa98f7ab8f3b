"""Oracle for the operators that feed the paged MLA decode (TEST
INFRASTRUCTURE ONLY): RMS norm, rotary positions, many-token cache append and
cache gather, in float64 numpy from their formulas.

The computed values come with a bound t on the 32-bit arithmetic's own error
(derived at each function); an output of a type is then right when it lies
between the roundings of y - t and y + t to that type, which is one value for
almost every y.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp4 as _fp4
from . import fp8 as _fp8

U = 2.0 ** -24          # half a unit in the last place of a 32-bit result, relative


# ---------------------------------------------------------------- rounding
def round_to(y: np.ndarray, kind: str) -> np.ndarray:
    """Nearest value of the type, ties to even (float64 in and out)."""
    y = np.asarray(y, dtype=np.float64)
    bits, emin, top = {"f32": (24, -126, np.finfo(np.float32).max), "f16": (11, -14, 65504.0),
                       "bf16": (8, -126, float.fromhex("0x1.fep127"))}[kind]
    _, e = np.frexp(np.where(np.isfinite(y), y, 1.0))
    unit = np.ldexp(1.0, np.maximum(e - 1, emin) - (bits - 1))
    with np.errstate(invalid="ignore"):
        r = np.round(y / unit) * unit
        r = np.where(np.abs(r) > top, np.copysign(np.inf, y), r)
    return np.where(np.isfinite(y), r, y)


def assert_rounded(got: np.ndarray, y: np.ndarray, t: np.ndarray, kind: str, label=""):
    got, y = np.asarray(got, dtype=np.float64), np.asarray(y, dtype=np.float64)
    lo, hi = round_to(y - t, kind), round_to(y + t, kind)
    ok = ((got >= lo) & (got <= hi)) | (np.isnan(got) & np.isnan(y))
    if not ok.all():
        i = np.unravel_index(int(np.argmin(ok)), ok.shape)
        raise AssertionError(f"{label}: {int((~ok).sum())} of {ok.size} off, first at {i}: "
                             f"{got[i]!r} not in [{lo[i]!r}, {hi[i]!r}]")


# ---------------------------------------------------------------- quantisers
def group_exponent(amax: np.ndarray, top: float) -> np.ndarray:
    """ceil(log2(amax / top)) clamped to [-127, 127], -127 for zero."""
    m, e = np.frexp(np.asarray(amax, dtype=np.float64) / top)
    e = np.where(m > 0.5, e, e - 1)
    return np.where(amax > 0, np.clip(e, -127, 127), -127)


def assert_quantised(codes: np.ndarray, e: np.ndarray, y: np.ndarray, t: np.ndarray, group: int,
                     kind: str, label=""):
    """codes: the values of the codes [..., n]; e: the groups' exponents.  y +-
    t: the values before rounding (n need not fill the last group)."""
    top, rnd = (448.0, _fp8._round_to_e4m3) if kind == "e4m3" else (6.0, _fp4._round_to_e2m1)
    n = y.shape[-1]
    pad = [(0, 0)] * (y.ndim - 1) + [(0, -n % group)]
    a, b = (np.pad(np.maximum(np.abs(y) + s * t, 0.0), pad).reshape(*y.shape[:-1], -1, group).max(-1)
            for s in (-1, 1))
    lo, hi = group_exponent(a, top), group_exponent(b, top)
    assert ((e >= lo) & (e <= hi)).all(), (label, "scales", np.argwhere((e < lo) | (e > hi))[:4])
    s = np.repeat(np.ldexp(1.0, np.asarray(e, dtype=np.int64)), group, axis=-1)[..., :n]
    lo, hi = rnd((y - t) / s), rnd((y + t) / s)
    ok = (codes >= lo) & (codes <= hi)
    assert ok.all(), (label, "codes", int((~ok).sum()), np.argwhere(~ok)[:4])


# ---------------------------------------------------------------- RMS norm
def rms_norm(x, residual=None, weight=None, eps=1e-6):
    """(h, y, t) of float64 rows.  t: h carries one rounding (U), its square
    two more and the sum of n of them, added in any tree of at least 32
    strands, at most n / 32 + 16 roundings; mean, eps and the root's argument
    another three.  The reciprocal root halves that error and adds two units
    of its own (it is accurate to 2 units in the last place), and two products
    follow.  Results below the normal range are off by at most two of its
    steps."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + residual
    n = h.shape[-1]
    y = h / np.sqrt((h * h).sum(-1, keepdims=True) / n + eps)
    if weight is not None:
        y = y * weight
    return h, y, np.abs(y) * (1 + (n / 32 + 16 + 6) / 2 + 4 + 2) * U + 2.0 ** -148


# ---------------------------------------------------------------- rotary positions
def rope_frequencies(dim, theta=1e6, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0):
    """Radians per position of each pair, and the scaling's own amplitude."""
    out = []
    for i in range(dim // 2):
        f = float(theta) ** (-2.0 * i / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "parts":
            turns = original * f / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            f = w * f + (1 - w) * f / factor
        elif scaling == "yarn":
            def pair(r):
                return dim * math.log(original / (2 * math.pi * r)) / (2 * math.log(theta))
            low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim - 1)
            w = 1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    return np.array(out), amplitude


def rope(x, positions, freq, amplitude=1.0, layout="pairs", transposed=False):
    """(y, t): x [tokens, ..., dim] turned.  t per pair (a, b): the angle is
    off by at most pi 2^-25 from its conversion to 32 bits (1.6 U) and pos *
    2^-52 turns from the table; the function by 2 U, the amplitude and its
    product by 2 U, the two products and their sum by 2 U more."""
    x = np.asarray(x, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64).reshape(-1, *([1] * (x.ndim - 1))) * freq
    c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude
    if transposed:
        s = -s
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "pairs" else (x[..., :h], x[..., h:])
    y, t = np.empty_like(x), np.empty_like(x)
    far = np.abs(np.asarray(positions, dtype=np.float64)).reshape(-1, *([1] * (x.ndim - 1)))
    # float64's own pos * freq is off by up to 2^-53 of the angle, relative
    bound = amplitude * (np.abs(a) + np.abs(b)) * (8 * U + far * (2.0 ** -52 * 2 * math.pi + freq * 2.0 ** -52))
    for dst, va, vb in ((y, a * c - b * s, a * s + b * c), (t, bound, bound)):
        if layout == "pairs":
            dst[..., 0::2], dst[..., 1::2] = va, vb
        else:
            dst[..., :h], dst[..., h:] = va, vb
    return y, t


# ---------------------------------------------------------------- cache rows
def slots_of(positions, requests, block_table, page_size, num_pages):
    """Each token's pool slot: -1 for a negative position, -2 for one without
    a slot."""
    B, max_pages = block_table.shape
    out = np.full(len(positions), -2, dtype=np.int64)
    for t, (p, r) in enumerate(zip(positions, requests)):
        if p < 0:
            out[t] = -1
        elif 0 <= r < B and p < max_pages * page_size:
            page = block_table[r, p // page_size]
            if 0 <= page < num_pages:
                out[t] = int(page) * page_size + p % page_size
    return out


def row_values(rows, positions, norm_weight=None, eps=1e-6, freq=None, amplitude=1.0, layout="pairs"):
    """(y, t) of the cache rows [tokens, 576] before their rounding."""
    rows = np.asarray(rows, dtype=np.float64)
    y, t = rows.copy(), np.zeros_like(rows)
    if norm_weight is not None:
        _, y[:, :512], t[:, :512] = rms_norm(rows[:, :512], weight=norm_weight, eps=eps)
    if freq is not None:
        y[:, 512:], t[:, 512:] = rope(rows[:, 512:], positions, freq, amplitude, layout)
    return y, t


def assert_cache_rows(raw, y, t, kv: str, label=""):
    """raw: the written rows, bf16 values [n, 576] or bytes [n, 594 | 324]."""
    if kv == "bf16":
        assert_rounded(raw, y, t, "bf16", label)
    elif kv == "fp8":
        assert_quantised(_fp8.e4m3_to_f64(raw[:, :576]), raw[:, 576:].astype(np.int64) - 127, y, t,
                         32, "e4m3", label)
    else:
        assert_quantised(_fp4.e2m1_to_f64(_fp4.unpack_codes(raw[:, :288])), raw[:, 288:].astype(np.int64) - 127, y, t, 16,
                         "e2m1", label)


def gather_rows(cache, slots, kv: str):
    """Rows of a paged cache (bytes or bf16 bits) as float64, rounded to bf16."""
    if kv == "bf16":
        bits = np.ascontiguousarray(cache).view(np.uint16).reshape(-1, 576)[slots]
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    enc = _fp8 if kv == "fp8" else _fp4
    return round_to(enc.dequant_rows(cache.reshape(-1, enc.ROW_BYTES)[slots]), "bf16")
