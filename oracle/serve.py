"""What stands around the paged cache, in fp64 (angles in extended precision): rotary frequencies
and positions, norms of heads, the rows of chunks.

Test infrastructure only (see the package docstring), written from the definitions.
"""
from __future__ import annotations

import math

import numpy as np

from . import paged


def freqs(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """(radians per token of each pair, magnitude)."""
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    if scaling == "by_pair":
        pair = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        b = b + 0.001 if a == b else b
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_pair":
            slow = min(max((i - a) / (b - a), 0.0), 1.0)
            f = f * (1 - slow) + f * slow / factor
        elif scaling == "by_turns":
            fast = min(max((f * original / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * fast + f * (1 - fast) / factor
        out.append(f)
    return np.array(out), 1 + 0.1 * math.log(factor) if scaling == "by_pair" and factor > 1 else 1.0


def norm(x, weight, offset, eps):
    """Heads [R, H, D]: x / sqrt(mean x^2 + eps) (weight + offset)."""
    x = np.asarray(x, np.float64)
    w = offset + (0.0 if weight is None else np.asarray(weight, np.float64))
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rope(x, place, f, layout, magnitude):
    """Heads [R, H, D] turned by the angles place[r] f[i]; also |a| + |b| of each element's pair,
    times the magnitude (what an error bound needs; |x| where nothing is turned)."""
    x = np.asarray(x, np.float64)
    y, size = x.copy(), np.abs(x)
    angle = np.asarray(place, np.longdouble)[:, None] * np.asarray(f, np.longdouble)[None]
    c, s = (np.asarray(g(angle), np.float64)[:, None] * magnitude for g in (np.cos, np.sin))
    half = len(f)
    i = np.arange(half)
    one, two = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size[..., one] = size[..., two] = (np.abs(a) + np.abs(b)) * abs(magnitude)
    return y, size


def chunk_rows(cu, lens, rows, max_len=None):
    """(request, visible tokens) of each row; request -1 and 0 tokens for rows of none."""
    req, sees = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    for b in range(len(lens)):
        for r in range(max(int(cu[b]), 0), min(int(cu[b + 1]), rows)):
            req[r], sees[r] = b, max(int(lens[b]) - int(cu[b + 1]) + r + 1, 0)
    return req, sees if max_len is None else np.minimum(sees, max_len)


def attend_chunk(q, k_cache, v_cache, table, cu, lens, scale=None, max_len=None):
    """As paged.attend, for the rows that cu and lens describe."""
    limit = table.shape[1] * k_cache.shape[2]
    req, sees = chunk_rows(cu, lens, q.shape[0], limit if max_len is None else max_len)
    return paged.attend(q, k_cache, v_cache, table, sees, req=req, scale=scale, max_len=max_len)
