"""Oracle — the 4-bit paged cache, attention over it and the page pool (TEST INFRASTRUCTURE ONLY).

Everything sequence by sequence and in float64, in plain loops: quantization by the NVFP4 oracle
(quant.py) with fixed tensor scales, pages filled token by token, attention as a textbook softmax,
the pool as lists.
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_decode, e4m3_decode
from .quant import nvfp4_quantize, nvfp4_unpack

PAGE = 64


class Cache:
    """Pages of the 4-bit cache as numpy arrays, one token and head written at a time."""

    def __init__(self, pages: int, heads: int, d: int, k_scale: float, v_scale: float):
        self.kp = np.zeros((pages, heads, PAGE, d // 2), np.uint8)
        self.ks = np.zeros((pages, heads, PAGE, d // 16), np.uint8)
        self.vp = np.zeros((pages, heads, PAGE // 2, d), np.uint8)
        self.vs = np.zeros((pages, heads, d // 16, PAGE), np.uint8)
        self.kt, self.vt = np.float32(k_scale), np.float32(v_scale)

    def append(self, k, v, start: int, row) -> None:
        """k, v [n, heads, d] float32 at positions start.. of the sequence with page list `row`."""
        if not len(k):
            return
        kc, ks, _ = nvfp4_quantize(k, self.kt)
        vc, vs, _ = nvfp4_quantize(v, self.vt)
        vc = nvfp4_unpack(vc)
        for i in range(len(k)):
            page, slot = row[(start + i) // PAGE], (start + i) % PAGE
            self.kp[page, :, slot] = kc[i]
            self.ks[page, :, slot] = ks[i]
            self.vs[page, :, :, slot] = vs[i]
            old = self.vp[page, :, slot // 2]
            self.vp[page, :, slot // 2] = (old & 0x0F) | (vc[i] << 4) if slot % 2 else (old & 0xF0) | vc[i]

    def read(self, n: int, row, start: int = 0):
        """Positions start .. start + n - 1: k, v [n, heads, d] float64."""
        at = np.arange(start, start + n)
        page, slot = np.asarray(row, dtype=np.int64)[at // PAGE], at % PAGE
        k = e2m1_decode(nvfp4_unpack(self.kp[page, :, slot]))
        k = k.reshape(*k.shape[:2], k.shape[2] // 16, 16) * e4m3_decode(self.ks[page, :, slot])[..., None]
        vb = self.vp[page, :, slot // 2]
        v = e2m1_decode(np.where((slot % 2)[:, None, None], vb >> 4, vb & 15))
        v = v.reshape(*v.shape[:2], v.shape[2] // 16, 16) * e4m3_decode(self.vs[page, :, :, slot])[..., None]
        return (k.reshape(vb.shape) * np.float64(self.kt), v.reshape(vb.shape) * np.float64(self.vt))


def attention(q, k, v, scale: float):
    """Causal attention of the last len(q) tokens: q [n, Hq, d], k, v [ctx, Hkv, d] ->
    out [n, Hq, d], lse [n, Hq], all float64."""
    n, hq, d = q.shape
    ctx, hkv, _ = k.shape
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    seen = np.arange(ctx)[None, :] <= np.arange(ctx - n, ctx)[:, None]
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        s = np.where(seen, (q[:, h] @ kh.T) * scale, -np.inf)
        m = s.max(axis=1, keepdims=True)
        w = np.exp(s - m)
        total = w.sum(axis=1, keepdims=True)
        out[:, h] = (w / total) @ vh
        lse[:, h] = (m + np.log(total))[:, 0]
    return out, lse


class Pool:
    """The page pool by its rules, on lists; a call that cannot be met raises and changes nothing."""

    def __init__(self, pages: int, seqs: int, width: int):
        self.refs, self.lens = [0] * pages, [0] * seqs
        self.table = [[-1] * width for _ in range(seqs)]

    @staticmethod
    def pages_of(n: int) -> int:
        return (n + PAGE - 1) // PAGE

    def _lowest(self, n: int):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        if len(free) < n:
            raise ValueError("too few free pages")
        return free[:n]

    def alloc(self, new_lens) -> None:
        need = [self.pages_of(b) - self.pages_of(a) for a, b in zip(self.lens, new_lens)]
        if any(b < a or self.pages_of(b) > len(self.table[0]) for a, b in zip(self.lens, new_lens)):
            raise ValueError("length")
        free = self._lowest(sum(need))
        for s, n in enumerate(need):
            for i in range(n):
                p = free.pop(0)
                self.table[s][self.pages_of(self.lens[s]) + i] = p
                self.refs[p] = 1

    def fork(self, src, dst):
        if len(set(dst)) < len(dst) or any(s == d or self.lens[d] for s, d in zip(src, dst)):
            raise ValueError("destination")
        lens = list(self.lens)
        free = self._lowest(sum(lens[s] % PAGE != 0 for s in src))
        moves = []
        for s, d in zip(src, dst):
            full = lens[s] // PAGE
            for i in range(full):
                self.table[d][i] = self.table[s][i]
                self.refs[self.table[s][i]] += 1
            if lens[s] % PAGE:
                p = free.pop(0)
                self.table[d][full] = p
                self.refs[p] = 1
                moves.append((self.table[s][full], p))
            else:
                moves.append((-1, -1))
            self.lens[d] = lens[s]
        return moves

    def free(self, seqs) -> None:
        for s in seqs:
            for i in range(self.pages_of(self.lens[s])):
                self.refs[self.table[s][i]] -= 1
                self.table[s][i] = -1
            self.lens[s] = 0

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        holes = [p for p in range(len(live)) if self.refs[p] == 0]
        moves = list(zip([p for p in live if p >= len(live)], holes))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, row in enumerate(self.table):
            for i in range(self.pages_of(self.lens[s])):
                row[i] = to.get(row[i], row[i])
        return moves
