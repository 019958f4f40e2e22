"""Oracle of the paged history cache: the page bookkeeping in plain Python, the
chunk attention (Eq. 2 for the last rows of a sequence, optionally through a
window with sinks) and the incremental encoder in float64.

TEST INFRASTRUCTURE ONLY, like oracle/hstu.py.
"""
from __future__ import annotations

import numpy as np

from . import hstu as O


class Pages:
    """Block tables, lengths and reference counts, one step at a time."""

    def __init__(self, num_pages: int, num_seqs: int, max_blocks: int, page_size: int):
        self.ps = page_size
        self.ref = [0] * num_pages
        self.table = [[-1] * max_blocks for _ in range(num_seqs)]
        self.len = [0] * num_seqs

    def blocks(self, n: int) -> int:
        return -(-n // self.ps)

    def reserve(self, seqs, counts):
        """Returns the copies [(source, copy, filled rows)] or None when refused."""
        if len(set(seqs)) != len(seqs) or any(not 0 <= s < len(self.len) for s in seqs):
            return None
        plan = []
        for s, c in zip(seqs, counts):
            n = self.len[s]
            if self.blocks(n + c) > len(self.table[s]):
                return None
            last = self.table[s][self.blocks(n) - 1] if n % self.ps else -1
            cow = c > 0 and n % self.ps != 0 and self.ref[last] > 1
            plan.append((s, c, last if cow else -1))
        need = sum(self.blocks(self.len[s] + c) - self.blocks(self.len[s]) + (src >= 0)
                   for s, c, src in plan)
        free = [p for p, r in enumerate(self.ref) if r == 0]
        if need > len(free):
            return None
        copies = []
        for s, c, src in plan:
            n = self.len[s]
            if src >= 0:
                page = free.pop(0)
                copies.append((src, page, n % self.ps))
                self.ref[page] = 1
                self.ref[src] -= 1
                self.table[s][self.blocks(n) - 1] = page
            for b in range(self.blocks(n), self.blocks(n + c)):
                page = free.pop(0)
                self.ref[page] = 1
                self.table[s][b] = page
            self.len[s] = n + c
        return copies

    def fork(self, src: int, dst: int):
        assert self.len[dst] == 0
        for b in range(self.blocks(self.len[src])):
            page = self.table[src][b]
            self.table[dst][b] = page
            if page >= 0:
                self.ref[page] += 1
        self.len[dst] = self.len[src]

    def release(self, seq: int, window: int = 0, sinks: int = 0):
        n = self.len[seq]
        for b in range(self.blocks(n)):
            # every event that a row at n or later sees: j < sinks or j > n - window
            if window and any(j < sinks or j > n - window
                              for j in range(b * self.ps, (b + 1) * self.ps)):
                continue
            if self.table[seq][b] >= 0:
                self.ref[self.table[seq][b]] -= 1
                self.table[seq][b] = -1
        if not window:
            self.len[seq] = 0

    def compact(self):
        """Returns the moves [(source, destination)]."""
        live = sum(r > 0 for r in self.ref)
        holes = [p for p in range(live) if self.ref[p] == 0]
        moves = [(p, holes.pop(0)) for p in range(live, len(self.ref)) if self.ref[p] > 0]
        to = dict(moves)
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return moves


def window_mask(n: int, c: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """Visibility [c, n] of the last c of n events."""
    i = np.arange(n - c, n)[:, None]
    j = np.arange(n)[None, :]
    vis = j <= i
    if window:
        vis &= (j > i - window) | (j < sinks)
    return vis


def chunk_attention(q, k, v, ts, rab_pos, rab_time, H: int, phi2: str = "silu", window: int = 0,
                    sinks: int = 0, parts: bool = False):
    """Eq. 2 for the last c = len(q) of n = len(k) events of one sequence, [c, H*64].
    With parts, also the pre-activations and weights [H, c, n]."""
    c, n = q.shape[0], k.shape[0]
    mask = window_mask(n, c, window, sinks)
    out = np.zeros((c, H * 64))
    ss, aa = np.zeros((H, c, n)), np.zeros((H, c, n))
    for h in range(H):
        cols = slice(h * 64, h * 64 + 64)
        s = q[:, cols] @ k[:, cols].T + O.rab_matrix(ts[n - c:], ts, np.arange(n - c, n), np.arange(n),
                                                     rab_pos[h], rab_time[h])
        a = O.attention_weights(s, mask, phi2, max(n, 1))
        out[:, cols] = a @ v[:, cols]
        ss[h], aa[h] = s, a
    return (out, ss, aa) if parts else out


def extend(state, x, ts, layers, cfg, window: int = 0, sinks: int = 0):
    """New events of one sequence through the stack.  `state`: per layer (K, V)
    arrays of the earlier events plus their times, as returned by the last call
    (None at the start).  Returns (Y, state)."""
    H, hv = cfg.num_heads, cfg.num_heads * 64
    if state is None:
        state = ([(np.zeros((0, hv)), np.zeros((0, hv))) for _ in layers], np.zeros(0, dtype=np.int64))
    kv, times = state
    times = np.concatenate([times, np.asarray(ts, dtype=np.int64)])
    cur, out = np.asarray(x, dtype=np.float64), []
    f = O._f64
    for layer, (k0, v0) in zip(layers, kv):
        u, v, q, k = O.projection(cur, f(layer.w1), f(layer.b1), H, 64, 64, cfg.phi1)
        k, v = np.concatenate([k0, k]), np.concatenate([v0, v])
        av = chunk_attention(q, k, v, times, f(layer.rab_pos), f(layer.rab_time), H, cfg.phi2, window,
                             sinks)
        cur, _ = O.output(cur, av, u, f(layer.w2), f(layer.b2), cfg.ln_eps, f(layer.ln_gamma),
                          f(layer.ln_beta))
        out.append((k, v))
    return cur, (out, times)
