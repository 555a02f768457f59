"""The context of block-by-block generation: block tables, rotary positions,
the append to the 8-bit paged cache and the attention over it, in plain
numpy and float64 (the tables in Python integers).

[Report] "DiffusionGemma Technical Report", Figure 4: finished blocks are
encoded and appended to the context that the next block attends to.  The
pages give no layout and no formulas beyond that; these are the definitions
include/dg.h states.

TEST INFRASTRUCTURE: part of the CPU oracle (see ``oracle/__init__``).
"""
from __future__ import annotations

import math

import numpy as np

from .step import decode_e4m3

PAGE = 64


def plan(table, held, free_list, free_count, add, release, rows):
    """Plan a batch; returns a dict of everything ``dg_context_plan`` writes.
    Inputs are lists (table a list of lists) and are not changed."""
    table = [list(r) for r in table]
    held, free_list = list(held), list(free_list)
    stack = free_list[:free_count]
    B, width = len(held), len(table[0])
    for r in range(B):
        if release is not None and release[r]:
            for j in range(-(-held[r] // PAGE)):
                stack.append(table[r][j])
            held[r] = 0
    for i, pg in enumerate(stack):
        free_list[i] = pg
    kept = len(stack)
    need = [-(-(h + a) // PAGE) - -(-h // PAGE) for h, a in zip(held, add)]
    code = 0
    if any(a < 0 or h + a > width * PAGE for h, a in zip(held, add)):
        code = 3
    elif sum(add) > rows:
        code = 2
    elif sum(need) > len(stack):
        code = 1
    out = dict(held=held, free_count=kept, status=code)
    positions, slots, runs, start, lens = [-1] * rows, [-1] * rows, [], [0], list(held)
    if code == 0:
        row = 0
        for r in range(B):
            for j in range(need[r]):
                table[r][-(-held[r] // PAGE) + j] = stack.pop()
            for p in range(held[r], held[r] + add[r]):
                pg, off = table[r][p // PAGE], p % PAGE
                positions[row], slots[row] = p, pg * PAGE + off
                if p == held[r] or off == 0:
                    runs.append([pg, row, off, 0])
                runs[-1][3] += 1
                row += 1
            lens[r] = held[r] + add[r]
            start.append(row)
    else:
        start = [0] * (B + 1)
    runs += [[-1, 0, 0, 0]] * (rows // PAGE + 2 * B - len(runs))
    out.update(table=table, free_list=free_list, free_next=len(stack), positions=positions, slots=slots, runs=runs,
               start=start, lens=lens)
    return out


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=4096):
    """(angle per position of each pair, magnitude)."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * j / rot)
    if scaling == "linear":
        f = f / factor
    if scaling != "parts":
        return f, 1.0

    def pair(turns):  # the pair that makes this many turns over the original length
        return rot * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
    low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
    ramp = np.clip((j - low) / max(high - low, 1e-3), 0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1


def rope(x, positions, freq, magnitude, interleaved):
    """x float64 [rows, heads, dim]; the first 2 len(freq) elements turned."""
    rot = 2 * len(freq)
    a = np.asarray(positions, np.float64)[:, None] * freq
    c, s = magnitude * np.cos(a)[:, None], magnitude * np.sin(a)[:, None]
    y = np.array(x, np.float64)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


E4M3 = np.sort(decode_e4m3(np.arange(127, dtype=np.uint8)))  # the finite magnitudes, 0 .. 448


def round_e4m3(x):
    """The nearest E4M3 values (ties to the even code), saturating."""
    m = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(E4M3, m)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - E4M3[lo], E4M3[hi] - m
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))  # code i of the sorted magnitudes is i
    return np.copysign(np.where(up, E4M3[hi], E4M3[lo]), x)


def scale_of(top):
    """The least power of two s with top <= 448 s, at least 2^-100; 1 for 0."""
    if top == 0:
        return 1.0
    e = math.ceil(math.log2(top / 448.0))
    while top > 448.0 * 2.0 ** e:
        e += 1
    while e > -100 and top <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -100)


def append(values, scales, x, runs):
    """Rows x [rows, heads, dim] into a cache held as values / scale (float64
    [pages, heads, PAGE, dim]) and scales [pages, heads]; both changed.
    Values that are not finite are stored as dg.h says."""
    for page, row, off, n in runs:
        if page < 0:
            continue
        for h in range(x.shape[1]):
            part = x[row:row + n, h]
            fin = np.isfinite(part)
            s = scale_of(float(np.max(np.abs(part[fin]), initial=0.0)))
            old = scales[page, h]
            if off > 0:
                s = max(s, old)
                if s > old:
                    values[page, h, :off] = round_e4m3(values[page, h, :off] * (old / s))
            scales[page, h] = s
            part = np.where(np.isnan(part), 0.0, part)
            values[page, h, off:off + n] = round_e4m3(part / s)


def attention(q, k, v, scale, causal, window):
    """One request: q [nq, heads, dim], k and v [n, kv heads, dim], all
    float64.  Returns (out, lse, sum w |v|, the largest sum |q_d k_d| scale)
    per row and head."""
    nq, hq, dim = q.shape
    n, hk, _ = k.shape
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full((nq, hq), -np.inf), np.zeros((nq, hq))
    for i in range(nq):
        pos = n - nq + i
        hi = pos + 1 if causal else n
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(hq):
            kk, vv = k[lo:hi, h // (hq // hk)], v[lo:hi, h // (hq // hk)]
            x = scale * (kk @ q[i, h])
            top = x.max()
            w = np.exp(x - top)
            out[i, h], mass[i, h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum()
            lse[i, h] = top + np.log(w.sum())
            size[i, h] = scale * np.max(np.abs(kk) @ np.abs(q[i, h]))
    return out, lse, mass, size
