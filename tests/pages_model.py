"""A paged cache in plain Python, and attention over it in 64 bits, for the tests."""
from __future__ import annotations

import numpy as np
import torch


class PagesModel:
    """One list of pages and one length per slot; K and V are CPU tensors."""

    def __init__(self, num_pages, max_seqs, width, page, K, V):
        self.page, self.width, self.num_pages = page, width, num_pages
        self.K, self.V = K.clone(), V.clone()
        self.rows = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.refs = [0] * num_pages

    def take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def append(self, seqs, Kn, Vn, counts=None):
        for i, s in enumerate(seqs):
            for t in range(Kn.shape[2] if counts is None else counts[i]):
                at = self.lens[s] % self.page
                if at == 0:
                    self.rows[s].append(self.take())
                p = self.rows[s][-1]
                self.K[p, :, at], self.V[p, :, at] = Kn[i, :, t], Vn[i, :, t]
                self.lens[s] += 1

    def _rows(self, source, a, b, n):
        self.K[b, :, :n], self.V[b, :, :n] = source.K[a, :, :n], source.V[a, :, :n]

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            full, rest = divmod(self.lens[a], self.page)
            new = self.rows[a][:full]
            for p in new:
                self.refs[p] += 1
            if rest:
                new = new + [self.take()]
                self._rows(self, self.rows[a][full], new[-1], rest)
            self.rows[b], self.lens[b] = new, self.lens[a]

    def copy(self, src, dst, source=None):
        source = source or self
        for a, b in zip(src, dst):
            new = [self.take() for _ in source.rows[a]]
            for j, (x, y) in enumerate(zip(source.rows[a], new)):
                self._rows(source, x, y, min(self.page, source.lens[a] - j * self.page))
            self.rows[b], self.lens[b] = new, source.lens[a]

    def free(self, seqs):
        for s in seqs:
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = [], 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        strays = [p for p in range(live, self.num_pages) if self.refs[p]]
        name = dict(zip(strays, holes))
        for a, b in name.items():
            self._rows(self, a, b, self.page)
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.rows = [[name.get(p, p) for p in r] for r in self.rows]
        return live

    def table(self):
        t = torch.full((len(self.rows), self.width), -1, dtype=torch.int32)
        for s, r in enumerate(self.rows):
            t[s, :len(r)] = torch.tensor(r, dtype=torch.int32)
        return t

    def check(self, pages, K, V):
        """The device's state and pools are this model's, bit for bit."""
        assert pages.lens.tolist() == self.lens
        assert pages.refs.tolist() == self.refs
        assert torch.equal(pages.table.cpu(), self.table())
        for got, want in ((K, self.K), (V, self.V)):
            bits = torch.int16 if got.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(got.cpu().view(bits), want.view(bits))


def attend64(Q, K, V, table, lens, seqs, scale, prefix_seq=0, prefix=0, causal=False):
    """(o, w, a): outputs in 64 bits [batch, q_heads, nq, d], sum of p |v| and the largest
    sum of |scale q k| over the tokens a query sees (for the error bounds).  CPU tensors."""
    B, Hq, nq, d = Q.shape
    page, H = K.shape[2], K.shape[1]
    G = Hq // H
    o = np.zeros((B, Hq, nq, d))
    w, a = np.zeros_like(o), np.zeros((B, Hq, nq))
    q = Q.double().numpy()
    for b, s in enumerate(seqs):
        if not 0 <= s < len(lens):
            continue
        n = lens[s]
        ids = [int(table[prefix_seq if t * page < prefix else s, t]) for t in range(-(-n // page))]
        for h in range(H):
            k = K[ids, h].reshape(-1, d)[:n].double().numpy()
            v = V[ids, h].reshape(-1, d)[:n].double().numpy()
            for i in range(nq):
                m = n - (nq - 1 - i) if causal else n
                if m <= 0:
                    continue
                x = q[b, h * G:(h + 1) * G, i]
                t = scale * (x @ k[:m].T)
                p = np.exp(t - t.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o[b, h * G:(h + 1) * G, i] = p @ v[:m]
                w[b, h * G:(h + 1) * G, i] = p @ np.abs(v[:m])
                a[b, h * G:(h + 1) * G, i] = (abs(scale) * (np.abs(x) @ np.abs(k[:m]).T)).max(-1)
    return o, w, a
