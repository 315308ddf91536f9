"""Plain 64-bit and loop-by-loop forms of the linear layer, the beam selection
and the page operations, written from their definitions in include/gad_attn.h."""
from __future__ import annotations

import math

import numpy as np
import torch


def activation(v: torch.Tensor, act: str) -> torch.Tensor:
    if act == "relu":
        return torch.where(v > 0, v, torch.where(v.isnan(), v, torch.zeros_like(v)))
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v * torch.sigmoid(v)
    assert act == "none"
    return v


def linear(x, w, bias=None, residual=None, act="none", out_dtype=None):
    """(y, bound) in float64: the exact result and how far a right kernel may be
    off.  The bound: the K products are summed in fp32, 16 at a time, each step
    off by at most 2^-23 of the magnitudes summed so far; the activations' slopes
    are below 1.13 and their fp32 evaluation is within 2^-21 of |v|; bias and
    residual are one fp32 addition each; the result is rounded once (half a step,
    eps / 2; below the normal range half the smallest step)."""
    out_dtype = out_dtype or x.dtype
    xd, wd = x.double(), w.double()
    v = xd @ wd.T
    mag = xd.abs() @ wd.abs().T
    err = (math.ceil(x.shape[1] / 16) + 8) * 2.0 ** -23 * mag
    if bias is not None:
        v = v + bias.double()
        err = err + 2.0 ** -24 * (v.abs() + err)
    y = activation(v, act)
    if act != "none":
        err = 1.13 * err + 2.0 ** -21 * (v.abs() + err)
    if residual is not None:
        y = y + residual.double()
        err = err + 2.0 ** -24 * (y.abs() + err)
    fi = torch.finfo(out_dtype)
    bound = err + fi.eps / 2 * (y.abs() + err) + fi.tiny * fi.eps / 2
    return y, bound


def beam(logits, scores, K, finished=None, pad=0):
    """Scores float64, parents and tokens [G, K] by sorting every candidate."""
    G, W, V = logits.shape
    out = np.full((G, K), -np.inf), np.full((G, K), -1, np.int64), np.full((G, K), -1, np.int64)
    x = logits.double().cpu().numpy()
    s = scores.double().cpu().numpy()
    fin = np.zeros((G, W), bool) if finished is None else finished.cpu().numpy().astype(bool)
    for g in range(G):
        key = np.full((W, V), -np.inf)
        for w in range(W):
            if fin[g, w]:
                key[w, pad] = s[g, w]
                continue
            r = x[g, w]
            if np.isnan(r).any() or np.isposinf(r).any() or not np.isfinite(r).any():
                continue
            m = r.max()
            key[w] = s[g, w] + (r - (m + math.log(math.fsum(np.exp(r - m)))))
        flat = np.where(np.isnan(key), -np.inf, key).reshape(-1)
        order = np.argsort(-flat, kind="stable")[:K]
        for i, c in enumerate(order):
            if flat[c] > -np.inf:
                out[0][g, i], out[1][g, i], out[2][g, i] = flat[c], g * W + c // V, c % V
    return out


class Pool:
    """Tables, lengths and reference counts as plain numpy arrays, changed by
    loops over rows and pages."""

    def __init__(self, rows, max_pages, page_size, num_pages):
        self.ps = page_size
        self.table = np.full((rows, max_pages), -1, np.int32)
        self.lens = np.full(rows, -1, np.int32)
        self.refs = np.zeros(num_pages, np.int32)

    def pages(self, r):
        return -(-int(self.lens[r]) // self.ps) if self.lens[r] > 0 else 0

    def _free(self):
        return [int(p) for p in np.nonzero(self.refs == 0)[0]]

    def fork(self, parent):
        """(copy_src, copy_dst, short of pages)"""
        old, lens, R = self.table, self.lens, len(self.lens)
        n_out = len(parent)
        table = np.full((n_out, old.shape[1]), -1, np.int32)
        new_lens = np.full(n_out, -1, np.int32)
        src, dst = np.full(n_out, -1, np.int32), np.full(n_out, -1, np.int32)
        for r in range(R):
            for j in range(self.pages(r)):
                self.refs[old[r, j]] -= 1
        seen, fresh = set(), []
        for r, p in enumerate(parent):
            if not 0 <= p < R or lens[p] < 0:
                continue
            n = self.pages(p)
            new_lens[r] = lens[p]
            table[r, :n] = old[p, :n]
            if lens[p] % self.ps and p in seen:
                n -= 1
                table[r, n] = -1
                fresh.append(r)
            seen.add(p)
            for j in range(n):
                self.refs[table[r, j]] += 1
        free = self._free()
        for r in fresh:
            p = parent[r]
            n = self.pages(p) - 1
            if not free:
                new_lens[r] -= new_lens[r] % self.ps
                continue
            page = free.pop(0)
            src[r], dst[r], table[r, n] = old[p, n], page, page
            self.refs[page] = 1
        short = sum(1 for r in fresh if dst[r] < 0)
        self.table, self.lens = table, new_lens
        return src, dst, short > 0

    def extend(self, L):
        """(positions, cache_loc, pool too small, row too small)"""
        R = len(self.lens)
        pos, loc = np.zeros((R, L), np.int64), np.full((R, L), -1, np.int64)
        need, over = [], False
        for r in range(R):
            if self.lens[r] < 0:
                continue
            pos[r] = int(self.lens[r]) + np.arange(L)
            n = -(-(int(self.lens[r]) + L) // self.ps)
            over |= n > self.table.shape[1]
            need += [(r, j) for j in range(self.pages(r), n)]
        free = self._free()
        short = len(need) > len(free)
        if not over and not short:
            for (r, j), page in zip(need, free):
                self.table[r, j] = page
                self.refs[page] = 1
            for r in range(R):
                if self.lens[r] >= 0:
                    loc[r] = self.table[r, pos[r] // self.ps].astype(np.int64) * self.ps + pos[r] % self.ps
                    self.lens[r] += L
        return pos.reshape(-1), loc.reshape(-1), short, over

    def free(self, leave):
        for r in np.nonzero(leave)[0]:
            for j in range(self.pages(r)):
                self.refs[self.table[r, j]] -= 1
            self.lens[r] = -1

    def compact(self, max_moves):
        used = int((self.refs != 0).sum())
        src = [p for p in range(used, len(self.refs)) if self.refs[p]][:max_moves]
        dst = [p for p in range(used) if not self.refs[p]][:len(src)]
        to = dict(zip(src, dst))
        for r in range(len(self.lens)):
            for j in range(self.pages(r)):
                self.table[r, j] = to.get(int(self.table[r, j]), self.table[r, j])
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        pad = [-1] * (max_moves - len(src))
        return np.array(src + pad, np.int32), np.array(dst + pad, np.int32), used
