"""Plain 64-bit models of rows of 4-bit values, of the rotation, of the reordering and of the
selection over beams, and inputs for them.

Attention over 4-bit rows has the tolerances derived in _cache_helpers: the rows' values are exact in
bf16 there as here, and the arithmetic behind them is the same.

Rotation: x cos - y sin in 32 bits (two products, one sum: 2^-22 of |x cos| + |y sin| at most), then
half a step of bf16, 2^-8 of the result; beside bf16's least normal value half of its least step, 2^-134.

Selection, value of a candidate: d = x - M is off by 2^-24 |d|; log2(e) d by another 2^-23 of it, the
exponential by 2^-22 of its value; a term e^d |d| is at most e^d max(|d|), and terms past |d| = 24 add
less than 2^-17 even if 2^17 of them sum up, so the sum's error is at most 24 * 2^-22.4 + 2^-22
< 2^-17.5 of it (sums in 32 bits: 32 terms of a thread, 8 shuffles and 8 warps, 2^-18).  The logarithm
in parts adds 2^-24.  Together below 2^-16; the value's rounding to 32 bits is 2^-24 of it."""
from __future__ import annotations

import types

import numpy as np
import torch

import _cache_helpers as C

ROW4 = 368
GRID4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
COLUMN_NIBBLE = np.array([0, 4, 1, 5, 2, 6, 3, 7])       # of columns 8 i .. 8 i + 7 in word i


def pack_rows4(x: torch.Tensor) -> np.ndarray:
    """bf16 [n, 512] -> packed rows, straight from the definition, value by value in 64 bits."""
    v = x.double().cpu().numpy()
    n = v.shape[0]
    rows = np.zeros((n, ROW4), dtype=np.uint8)
    codes = np.zeros((n, 448), dtype=np.uint64)
    for g in range(14):
        part = v[:, 32 * g:32 * g + 32]
        for i in range(n):
            if not np.isfinite(part[i]).all():
                rows[i, 224 + g] = 255
                continue
            top = np.abs(part[i]).max()
            byte = 127
            if top > 0:
                e = -140
                while top > 6.0 * 2.0 ** e:
                    e += 1
                byte = min(max(e + 127, 1), 254)
            rows[i, 224 + g] = byte
            y = np.abs(part[i]) / 2.0 ** (byte - 127.0)
            hi = np.clip(np.searchsorted(GRID4, y), 1, 7)
            lo = hi - 1
            dlo, dhi = y - GRID4[lo], GRID4[hi] - y
            pick = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
            codes[i, 32 * g:32 * g + 32] = pick + np.where(np.signbit(part[i]), 8, 0)
    words = np.zeros((n, 56), dtype=np.uint64)
    for k in range(8):
        words |= codes[:, k::8] << np.uint64(4 * COLUMN_NIBBLE[k])
    rows[:, :224] = words.astype("<u4").view(np.uint8).reshape(n, 224)
    rows[:, 240:] = x[:, 448:].contiguous().cpu().view(torch.int16).numpy().view(np.uint8).reshape(n, 128)
    return rows


def dequantize4(rows: np.ndarray):
    """uint8 [n, >= 368] -> (nope [n, 448], rope [n, 64]) in 64 bits."""
    rows = np.ascontiguousarray(rows[:, :ROW4])
    n = rows.shape[0]
    words = np.ascontiguousarray(rows[:, :224]).view("<u4")
    nope = np.zeros((n, 448))
    for k in range(8):
        c = (words >> np.uint32(4 * COLUMN_NIBBLE[k])) & 15
        nope[:, k::8] = np.where(c >= 8, -1.0, 1.0) * GRID4[c & 7]
    s = rows[:, 224:238].astype(np.float64)
    scale = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    nope = (nope.reshape(n, 14, 32) * scale[:, :, None]).reshape(n, 448)
    bits = np.ascontiguousarray(rows[:, 240:368]).view("<u2").astype(np.uint32) << 16
    return nope, bits.view(np.float32).astype(np.float64)


def random_pool4(num_pages: int, page: int, seed: int, stride: int = ROW4, lead: int = 0, mult: float = 1.0):
    """A pool of rows of normal values on the GPU, in an allocation filled with 0xA5 (lead: bytes
    before the first row, a multiple of 16)."""
    rng = np.random.default_rng(seed)
    n = num_pages * page
    nibbles = rng.choice(16, size=(n, 448), p=np.repeat([.1, .2, .2, .15, .15, .1, .07, .03], 2)[
        np.argsort(np.concatenate([np.arange(8) * 2, np.arange(8) * 2 + 1]), kind="stable")] / 2)
    words = np.zeros((n, 56), dtype=np.uint64)
    for k in range(8):
        words |= nibbles[:, k::8].astype(np.uint64) << np.uint64(4 * COLUMN_NIBBLE[k])
    rows = np.zeros((n, ROW4), dtype=np.uint8)
    rows[:, :224] = words.astype("<u4").view(np.uint8).reshape(n, 224)
    rows[:, 224:238] = rng.integers(125, 128, size=(n, 14)) + int(round(np.log2(mult)))
    rows[:, 238:240] = rng.integers(0, 256, size=(n, 2))
    rope = torch.as_tensor(rng.standard_normal((n, 64)) * mult, dtype=torch.float32).to(torch.bfloat16)
    rows[:, 240:] = rope.view(torch.int16).numpy().view(np.uint8).reshape(n, 128)
    store = torch.full((lead + n * stride,), 0xA5, dtype=torch.uint8, device="cuda")
    pool = store[lead:].view(n, stride)
    pool[:, :ROW4] = torch.as_tensor(rows).cuda()
    return pool


def chunk_reference4(*args, **kw):
    """_cache_helpers.chunk_reference over 4-bit rows."""
    row, oracle = C.ROW, C.O
    C.ROW, C.O = ROW4, types.SimpleNamespace(dequantize_rows=dequantize4)
    try:
        return C.chunk_reference(*args, **kw)
    finally:
        C.ROW, C.O = row, oracle


# ---------------------------------------------------------------- rotation
def rotary_table(positions: int, seed: int = 0) -> torch.Tensor:
    """fp32 [positions, 64]: rotations as a model has them, in 64 bits first."""
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(32) / 32.0)
    return torch.as_tensor(np.concatenate([np.cos(a), np.sin(a)], axis=1), dtype=torch.float32).cuda()


def rotate64(x: torch.Tensor, turn: torch.Tensor, interleaved: bool):
    """x [..., 64], turn [..., 64] -> rotated values and their tolerance, in 64 bits."""
    x, c, s = x.double(), turn[..., :32].double(), turn[..., 32:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, a * s + b * c
    tu, tv = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    out, mag = torch.empty_like(x), torch.empty_like(x)
    if interleaved:
        out[..., 0::2], out[..., 1::2], mag[..., 0::2], mag[..., 1::2] = u, v, tu, tv
    else:
        out[..., :32], out[..., 32:], mag[..., :32], mag[..., 32:] = u, v, tu, tv
    return out, 2.0 ** -8 * out.abs() + 2.0 ** -21 * mag + 2.0 ** -134


# ---------------------------------------------------------------- reordering
def reorder_model(model: C.PageModel, parents):
    """The definition of smla_cache_reorder on a page model, one row at a time."""
    R, page = len(model.table), model.page
    pages = len(model.ref)
    old, lens = [list(r) for r in model.table], list(model.lens)
    parents = [p if 0 <= p < R else -1 for p in parents]
    first = {}
    for r, p in enumerate(parents):
        if p >= 0:
            first.setdefault(p, r)
    for r in range(R):
        if r not in first:
            for p in old[r]:
                if 0 <= p < pages:
                    model.ref[p] -= 1
    width = len(old[0])
    length = [min(max(L, 0), width * page) for L in lens]
    fresh = {}
    for r, p in enumerate(parents):              # pages are taken before any count changes
        if p >= 0 and first[p] != r and length[p] % page and 0 <= old[p][length[p] // page] < pages:
            fresh[r] = model._take()
    for r, p in enumerate(parents):
        if p < 0 or fresh.get(r) == -1:
            model.table[r], model.lens[r] = [-1] * width, 0
        elif first[p] == r:
            model.table[r], model.lens[r] = list(old[p]), lens[p]
        else:
            L = length[p]
            full, rem = L // page, L % page
            row = [-1] * width
            for i in range(full):
                row[i] = old[p][i]
                if 0 <= row[i] < pages:
                    model.ref[row[i]] += 1
            if rem:
                row[full] = fresh.get(r, old[p][full])
                if r in fresh:
                    model.copies.append((old[p][full], fresh[r], rem))
            model.table[r], model.lens[r] = row, L


# ---------------------------------------------------------------- selection
def select_reference(logits, scores, num_out, finished=None, end_token=0):
    """(parents, tokens, values) in 64 bits, ties to the lower beam and token."""
    x = logits.detach().cpu().double().numpy()
    G, K = scores.shape
    c = scores.detach().cpu().double().numpy()
    parents, tokens = np.full((G, num_out), -1), np.full((G, num_out), -1)
    values = np.full((G, num_out), -np.inf)
    for g in range(G):
        rows, toks, vals = [], [], []
        for j in range(K):
            r = g * K + j
            if not np.isfinite(c[g, j]):
                continue
            if finished is not None and bool(finished[r]):
                rows.append(np.array([r])), toks.append(np.array([end_token])), vals.append(np.array([c[g, j]]))
                continue
            v = x[r]
            if np.isnan(v).any() or np.isposinf(v).any() or np.isneginf(v).all():
                continue
            d = v - v.max()
            at = np.flatnonzero(~np.isneginf(v))
            # only a row's num_out largest can be among the group's
            at = at[np.lexsort((at, -v[at]))[:num_out]]
            rows.append(np.full(at.size, r)), toks.append(at)
            vals.append((c[g, j] + d[at]) - np.log(np.exp(d).sum()))     # equal but for rounding: equal
        if rows:
            rows, toks, vals = np.concatenate(rows), np.concatenate(toks), np.concatenate(vals)
            order = np.lexsort((toks, rows, -vals))[:num_out]
            k = order.size
            parents[g, :k], tokens[g, :k], values[g, :k] = rows[order], toks[order], vals[order]
    return parents, tokens, values
