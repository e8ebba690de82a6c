"""fp64 oracle for the operators around the paged latent cache: TEST
INFRASTRUCTURE (imported only by tests/).  Plain loops over tokens, rows and
pages, from the definitions; shares no code with the product.

Rotary positions: pair i of 32 turns by pos * f_i; f_i = theta^(-2i/64), "linear"
divides it by a factor, "yarn" blends both by wavelength (YaRN, arXiv 2309.00071,
section 3.2).

8-bit pages: a page (64 tokens, one latent head) holds e4m3 values and a scale 2^e,
e the least whole number with amax <= 448 * 2^e; new rows join a page that
already holds some under the larger of its scale and theirs.
"""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE, D_QK, D_V = 64, 576, 512
MIN_EXP, MAX_EXP = -100, 119


def frequencies(theta=10000.0, scaling="none", factor=1.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0):
    f = np.array([theta ** (-2.0 * i / 64) for i in range(32)])
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        at = [64 * math.log(original_max_position / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (beta_fast, beta_slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), 63)
        for i in range(32):
            r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f[i] = f[i] * (1 - r) + f[i] / factor * r
    return f


def rotate(x, pos, interleaved=True, amplitude=1.0, transpose=False, **freq):
    """x [T, ..., 64] fp64, pos [T] -> the same, rotated."""
    x = np.asarray(x, dtype=np.float64)
    y = np.empty_like(x)
    f = frequencies(**freq)
    for t in range(x.shape[0]):
        for i in range(32):
            ang = math.fmod(int(pos[t]) * f[i], 2 * math.pi)
            c, s = math.cos(ang) * amplitude, math.sin(ang) * amplitude
            if transpose:
                s = -s
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            y[t, ..., a] = x[t, ..., a] * c - x[t, ..., b] * s
            y[t, ..., b] = x[t, ..., a] * s + x[t, ..., b] * c
    return y


def scale_of(amax: float) -> float:
    if amax == 0:
        return 2.0 ** MIN_EXP
    m, e = math.frexp(amax)          # amax = m 2^e, 0.5 <= m < 1;  448 = 0.875 * 2^9
    return 2.0 ** max(MIN_EXP, min(MAX_EXP, e - 9 + (1 if m > 0.875 else 0)))


def e4m3(x):
    """fp64 array -> the nearest e4m3 values (ties to even), as fp64; what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    with np.errstate(all="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
        step = np.exp2(e - 3)
        y = np.sign(x) * np.minimum(np.round(a / step) * step, 448.0)  # np.round: half to even
    return np.where(np.isfinite(x), y, np.nan)


def append(c_kv, k_pe, off, bt, lens, pool, scales=None, rope=None):
    """pool [num_blocks, 64, 576] fp64 (stored values; e4m3 units where scales is
    given), changed in place with scales.  Returns {(page): exact new rows} for
    comparisons: dict page -> (first row, fp64 rows before rounding)."""
    seen = {}
    for b in range(len(lens)):
        n, L = int(off[b + 1] - off[b]), int(lens[b])
        if n <= 0:
            continue
        pos = np.arange(L - n, L)
        pe = np.asarray(k_pe[off[b]:off[b + 1]], dtype=np.float64)
        if rope is not None:
            pe = rotate(pe, pos, **rope)
        rows = np.concatenate([np.asarray(c_kv[off[b]:off[b + 1]], dtype=np.float64), pe], axis=1)
        for page in range((L - n) // PAGE, (L + PAGE - 1) // PAGE):
            mine = pos // PAGE == page
            phys, first, x = int(bt[b][page]), int(pos[mine][0]) % PAGE, rows[mine]
            seen[phys] = (first, x)
            if scales is None:
                pool[phys, first:first + len(x)] = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
                continue
            fin = np.abs(x[np.isfinite(x)])
            s = scale_of(float(fin.max()) if fin.size else 0.0)
            if first > 0:
                s = max(s, float(scales[phys]))
                if s > scales[phys]:
                    pool[phys, :first] = e4m3(pool[phys, :first] * (float(scales[phys]) / s))
            pool[phys, first:first + len(x)] = e4m3(x / s)
            scales[phys] = s
    return seen


# ------------------------------------------------------------------ pages
def pages_of(n):
    return (n + PAGE - 1) // PAGE


def fork(parents, children, bt, lens, refs):
    """Books (numpy int arrays) changed in place; returns the (src, dst) page copies."""
    copies = []
    before = lens.copy()
    free = [i for i in range(len(refs)) if refs[i] == 0]
    named = set()
    for p, c in zip(parents, children):
        again, _ = c in named, named.add(c)
        if again or not (0 <= p < len(lens) and 0 <= c < len(lens)) or before[c] != 0:
            continue
        L = int(before[p])
        if L % PAGE:
            if not free:
                continue
            dst = free.pop(0)
            copies.append((int(bt[p, L // PAGE]), dst))
            bt[c, L // PAGE] = dst
            refs[dst] = 1
        for j in range(L // PAGE):
            bt[c, j] = bt[p, j]
            refs[bt[p, j]] += 1
        lens[c] = L
    return copies


def free(rows, bt, lens, refs):
    for r in rows:
        if 0 <= r < len(lens):
            for j in range(pages_of(int(lens[r]))):
                refs[bt[r, j]] -= 1
                bt[r, j] = -1
            lens[r] = 0


def compact(bt, lens, refs):
    live = int((refs > 0).sum())
    dst = [i for i in range(live) if refs[i] <= 0]
    src = [i for i in range(live, len(refs)) if refs[i] > 0]
    to = dict(zip(src, dst))
    for s, d in to.items():
        refs[d], refs[s] = refs[s], 0
    for b in range(len(lens)):
        for j in range(pages_of(int(lens[b]))):
            bt[b, j] = to.get(int(bt[b, j]), bt[b, j])
    return list(to.items())
