"""Plain 64-bit models of the paged-cache calls, and inputs for them.

Chunk attention tolerance, for one (token, head) row, from what the arithmetic rounds:
  - scores: 512 products summed in 32 bits, each of at most 512 additions off by 2^-23 of
    the running magnitude sum (truncating accumulation), so a score is off by at most
        delta = 2^-14 * scale * max_s sum_c |q_c| |k_sc|
    (512 * 2^-23 = 2^-14), plus 2^-20 of the cap (tanh through exp and a reciprocal) and
    2^-22 of the largest |bias| (two 32-bit roundings, doubled);
  - exp and log in 32 bits: 2^-20 of the sum, 2^-22 of |lse|;
  - the weights in bf16 before the value product: half a step, 2^-8 of each weight, which
    moves out by at most 2^-8 D, D = sum_s w_s |v_s - out|; a score error moves it by at
    most 2 delta D;
  - out in bf16: half a step, 2^-8 |out|.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle.mla_oracle as O

SCALE = 1.0 / np.sqrt(512.0)
ROW = 584


def pack_rows(x: torch.Tensor) -> np.ndarray:
    """bf16 [n, 512] -> packed rows, straight from the definition, value by value in 64 bits."""
    v = x.double().cpu().numpy()
    n = v.shape[0]
    rows = np.zeros((n, ROW), dtype=np.uint8)
    finite = [(O.E4M3_TABLE[b], b) for b in range(0x7F)]      # 0 .. 448, ascending
    grid = np.array([f for f, _ in finite])
    for g in range(7):
        part = v[:, 64 * g:64 * g + 64]
        mag = np.where(np.isfinite(part), np.abs(part), 0.0)
        top = mag.max(axis=1, initial=0.0)
        byte = np.full(n, 127)
        for i in range(n):
            if top[i] > 0:
                e = -140
                while top[i] > 448.0 * 2.0 ** e:
                    e += 1
                byte[i] = min(max(e + 127, 1), 254)
        y = mag / 2.0 ** (byte - 127.0)[:, None]
        # nearest of the grid, ties to the even byte
        hi = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
        lo = hi - 1
        dlo, dhi = y - grid[lo], grid[hi] - y
        pick = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
        code = pick.astype(np.uint8) | np.where(np.signbit(part), 0x80, 0).astype(np.uint8)
        code = np.where(np.isfinite(part), code, 0x7F)
        rows[:, 64 * g:64 * g + 64] = code
        rows[:, 448 + g] = byte
    rows[:, 456:] = x[:, 448:].contiguous().cpu().view(torch.int16).numpy().view(np.uint8).reshape(n, 128)
    return rows


def random_pool(num_pages: int, page: int, seed: int, stride: int = ROW, lead: int = 0, mult: float = 1.0):
    """A pool of random rows on the GPU; stride > 584 and lead (bytes before the first row)
    give a strided view into a larger allocation filled with 0xA5."""
    rng = np.random.default_rng(seed)
    n = num_pages * page
    x = torch.as_tensor(rng.standard_normal((n, 512)) * mult, dtype=torch.float32).to(torch.bfloat16)
    from sparse_mla_decode_03_gb300 import workloads as W
    rows = torch.cat([W._quantise_block(x[:, :448].float(), 0xFF),
                      x[:, 448:].contiguous().view(torch.uint8).view(n, 128)], dim=1)
    store = torch.full((lead + n * stride,), 0xA5, dtype=torch.uint8, device="cuda")
    pool = store[lead:].view(n, stride)
    pool[:, :ROW] = rows.cuda()
    return pool


def tables(lens, page: int, num_pages: int, seed: int, extra: int = 1):
    """Block table int32 [B, width] with distinct shuffled pages, on the host."""
    rng = np.random.default_rng(seed + 1)
    need = [-(-max(int(L), 0) // page) for L in lens]
    width = max(need + [1]) + extra
    assert sum(need) <= num_pages
    order = rng.permutation(num_pages)
    t = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda")


def chunk_reference(q, pool, table, page, cu_q, lens, scale=SCALE, cap=0.0, slopes=None, begin=None, end=None):
    """out, lse and their tolerances, float64 on the GPU: one token at a time.  Rows outside
    every sequence are NaN."""
    T, H, _ = q.shape
    f = dict(dtype=torch.float64, device="cuda")
    out = torch.full((T, H, 448), float("nan"), **f)
    lse = torch.full((T, H), float("nan"), **f)
    tol_out, tol_lse = torch.zeros((T, H, 448), **f), torch.zeros((T, H), **f)
    num_rows = pool.shape[0]
    for b in range(len(lens)):
        L = int(lens[b])
        pos_all = np.arange(max(L, 0))
        page_of = pos_all // page
        inside = page_of < table.shape[1]
        phys = np.where(inside, table[b, np.minimum(page_of, table.shape[1] - 1)], -1).astype(np.int64)
        row = phys * page + pos_all % page
        mapped = (phys >= 0) & (row < num_rows)
        data = pool[torch.as_tensor(np.where(mapped, row, 0), device="cuda")][:, :ROW].cpu().numpy()
        nope, rope = O.dequantize_rows(data) if L > 0 else (np.zeros((0, 448)), np.zeros((0, 64)))
        k = torch.as_tensor(np.concatenate([nope, rope], axis=1), **f)
        mapped_t = torch.as_tensor(mapped, device="cuda")
        for t in range(int(cu_q[b]), int(cu_q[b + 1])):
            pos = L - (int(cu_q[b + 1]) - t)
            lo = max(0, int(begin[t])) if begin is not None else 0
            hi = min(L, int(end[t])) if end is not None else pos + 1
            sel = torch.zeros(max(L, 0), dtype=torch.bool, device="cuda")
            if hi > lo:
                sel[lo:hi] = True
            sel &= mapped_t
            if not bool(sel.any()):
                out[t] = 0
                lse[t] = float("-inf")
                continue
            ks = k[sel]
            qt = q[t].double()
            x = scale * (qt @ ks.T)
            delta = 2.0 ** -14 * scale * (qt.abs() @ ks.abs().T).amax(dim=1)
            if cap:
                x = cap * torch.tanh(x / cap)
                delta = delta + 2.0 ** -20 * cap
            if slopes is not None:
                away = (torch.arange(max(L, 0), **f)[sel] - pos).abs()
                bias = slopes.double()[:, None] * away
                x = x - bias
                delta = delta + 2.0 ** -22 * bias.abs().amax(dim=1)
            z = torch.logsumexp(x, dim=1)
            w = torch.exp(x - z[:, None])
            v = ks[:, :448]
            o = w @ v
            D = torch.stack([w[h] @ (v - o[h]).abs() for h in range(H)])
            out[t], lse[t] = o, z
            tol_lse[t] = delta + 2.0 ** -20 + 2.0 ** -22 * z.abs()
            tol_out[t] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * delta[:, None]) * D + 1e-30
    return out, lse, tol_out, tol_lse


def check_chunk(got, ref):
    """got (out, lse) against chunk_reference's answer, on the rows that belong to a sequence."""
    out, lse = got
    o, z, to, tz = ref
    rows = ~torch.isnan(z)
    g = out.double()
    assert torch.isfinite(g[rows]).all(), "non-finite output"
    d = (g - o).abs()[rows]
    worst = (d / to[rows].clamp_min(1e-30)).max().item() if d.numel() else 0.0
    assert (d <= to[rows]).all(), f"out: worst error / tolerance {worst:.3g}"
    zl = lse.double()
    assert torch.equal(torch.isneginf(zl[rows]), torch.isneginf(z[rows])), "-inf pattern of lse"
    fin = rows & ~torch.isneginf(z)
    dz = (zl - z).abs()[fin]
    assert (dz <= tz[fin]).all(), f"lse: worst error / tolerance {(dz / tz[fin]).max().item():.3g}"


# ---------------------------------------------------------------- page bookkeeping, in Python
class PageModel:
    """ref_count, block_table and kv_lens as lists; the calls' definitions, one step at a time."""

    def __init__(self, ref, table, lens, page):
        self.ref, self.table, self.lens, self.page = list(map(int, ref)), [list(map(int, r)) for r in table], \
            list(map(int, lens)), page
        self.copies = []       # (from page, to page, rows) in the order made

    def _take(self):
        for p, c in enumerate(self.ref):
            if c == 0:
                self.ref[p] = 1
                return p
        return -1

    def free(self, rows):
        for r in rows:
            for i, p in enumerate(self.table[r]):
                if p >= 0:
                    self.ref[p] -= 1
                    self.table[r][i] = -1
            self.lens[r] = 0

    def reserve(self, target):
        for r, t in enumerate(target):
            for i in range(min(-(-int(t) // self.page), len(self.table[r]))):
                if self.table[r][i] < 0:
                    self.table[r][i] = self._take()

    def fork(self, parents, children):
        fresh = []
        for p, c in zip(parents, children):   # pages are taken before any count changes
            fresh.append(self._take() if self.lens[p] % self.page else -2)
        for p, c, f in zip(parents, children, fresh):
            L = self.lens[p] if f != -1 else 0
            full, rem = L // self.page, L % self.page
            row = [-1] * len(self.table[c])
            for i in range(full):
                row[i] = self.table[p][i]
                if row[i] >= 0:
                    self.ref[row[i]] += 1
            if rem:
                row[full] = f
                self.copies.append((self.table[p][full], f, rem))
            self.table[c], self.lens[c] = row, L

    def compact(self):
        used = [p for p, c in enumerate(self.ref) if c > 0]
        n = len(used)
        holes = [p for p in range(n) if self.ref[p] == 0]
        moves = list(zip([p for p in used if p >= n], holes))
        to = dict(moves)
        for s, d in moves:
            self.ref[d], self.ref[s] = self.ref[s], 0
            self.copies.append((s, d, self.page))
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return n, len(moves)


def check_pages(model, ref, table, lens):
    assert ref.cpu().tolist() == model.ref
    assert table.cpu().tolist() == model.table
    if lens is not None:
        assert lens.cpu().tolist() == model.lens
