"""The paged cache's bookkeeping and copies in plain Python lists and torch
indexing on the host, one entry at a time: what the GPU calls are compared with."""
import numpy as np
import torch

from copy_reduce_amd import TB_CACHE_BUSY, TB_CACHE_RANGE, TB_CACHE_SHARED, TB_CACHE_SHORT, TB_CACHE_TWICE


class Model:
    def __init__(self, num_pages, page_tokens, max_seqs, max_pages, kv, layout):
        self.P, self.pt, self.S, self.MP, self.layout = num_pages, page_tokens, max_seqs, max_pages, layout
        self.kv = kv.clone()           # [npools, P, ...] on the host
        self.table = [[0] * max_pages for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.refs = [0] * num_pages
        self.stack = list(range(num_pages - 1, -1, -1))
        self.free_above = {}           # what the stack's array holds above its top
        self.flags = 0

    def npg(self, n):
        return -(-n // self.pt)

    def by_token(self):
        return self.kv if self.layout == "token" else self.kv.transpose(2, 3)

    def pop(self):
        page = self.stack.pop()
        self.free_above[len(self.stack)] = page
        return page

    def push(self, page):
        self.free_above.pop(len(self.stack), None)
        self.stack.append(page)

    def copy_pages(self, dst, src, other=None):
        o = self if other is None else other
        was = o.kv.clone()
        for d, s in zip(dst, src):
            if 0 <= d < self.P and 0 <= s < o.P:
                self.kv[:, d] = was[:, s]

    def append(self, rows, seqs, positions, index=None):
        kv = self.by_token()
        for i, (q, p) in enumerate(zip(seqs, positions)):
            x = i if index is None else index[i]
            if q < 0:
                continue
            if q >= self.S or not 0 <= p < self.lens[q] or not 0 <= x < rows.shape[1]:
                self.flags |= TB_CACHE_RANGE
                continue
            page = self.table[q][p // self.pt]
            if self.refs[page] > 1:
                self.flags |= TB_CACHE_SHARED
                continue
            kv[:, page, p % self.pt] = rows[:, x]

    def fork(self, parents, children):
        before, todo, seen = list(self.lens), [], set()
        for p, c in zip(parents, children):
            if p < 0 or c < 0:
                continue
            if p >= self.S or c >= self.S:
                if c < self.S:
                    seen.add(c)
                self.flags |= TB_CACHE_RANGE
            elif c in seen:
                self.flags |= TB_CACHE_TWICE
            else:
                seen.add(c)
                if p == c or before[c]:
                    self.flags |= TB_CACHE_BUSY
                else:
                    todo.append((p, c))
        if sum(before[p] % self.pt > 0 for p, _ in todo) > len(self.stack):
            self.flags |= TB_CACHE_SHORT
            return
        kv = self.by_token()
        for p, c in todo:
            n = before[p]
            self.lens[c] = n
            for j in range(n // self.pt):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            if n % self.pt:
                page = self.pop()
                self.table[c][n // self.pt] = page
                self.refs[page] = 1
                kv[:, page, :n % self.pt] = kv[:, self.table[p][n // self.pt], :n % self.pt]

    def resize(self, seqs, lens):
        todo, seen, freed = [], set(), []
        for q, n in zip(seqs, lens):
            if q < 0:
                continue
            if q >= self.S or not 0 <= n <= self.MP * self.pt:
                self.flags |= TB_CACHE_RANGE
                seen.add(q)
            elif q in seen:
                self.flags |= TB_CACHE_TWICE
            else:
                seen.add(q)
                todo.append((q, n, self.npg(self.lens[q])))
        for q, n, had in todo:
            for j in range(self.npg(n), had):
                page = self.table[q][j]
                self.refs[page] -= 1
                if not self.refs[page]:
                    freed.append(page)
        for page in sorted(freed, reverse=True):
            self.push(page)
        short = sum(max(0, self.npg(n) - had) for _, n, had in todo) > len(self.stack)
        if short:
            self.flags |= TB_CACHE_SHORT
        for q, n, had in todo:
            if self.npg(n) > had:
                if short:
                    continue
                for j in range(had, self.npg(n)):
                    page = self.pop()
                    self.table[q][j] = page
                    self.refs[page] = 1
            self.lens[q] = n

    def compact(self):
        used = [p for p in range(self.P) if self.refs[p]]
        live = len(used)
        holes = [p for p in range(live) if not self.refs[p]]
        to = dict(zip([p for p in used if p >= live], holes))
        for a, b in to.items():
            self.kv[:, b] = self.kv[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for q in range(self.S):
            for j in range(self.npg(self.lens[q])):
                self.table[q][j] = to.get(self.table[q][j], self.table[q][j])
        self.stack = list(range(self.P - 1, live - 1, -1))

    def state(self, like):
        """The state tensor; words that are no part of the state are taken from `like`."""
        out = np.array(like, dtype=np.int64)
        a = self.S * self.MP
        for q in range(self.S):
            n = self.npg(self.lens[q])
            out[q * self.MP:q * self.MP + n] = self.table[q][:n]
        out[a:a + self.S] = self.lens
        out[a + self.S:a + self.S + self.P] = self.refs
        f = a + self.S + self.P
        out[f:f + len(self.stack)] = self.stack
        out[f + self.P], out[f + self.P + 1] = len(self.stack), self.flags
        return out

    def check(self, cache, what=""):
        got = cache.state.cpu().numpy().astype(np.int64)
        want = self.state(got)
        bad = np.nonzero(got != want)[0]
        assert bad.size == 0, f"{what}: state word {bad[0]} is {got[bad[0]]}, not {want[bad[0]]} ({bad.size} differ)"
        for i, p in enumerate(cache.pools):
            assert torch.equal(p.cpu().view(torch.uint8), self.kv[i].view(torch.uint8)), f"{what}: pool {i}"

    def context(self, pool, q, head):
        """[lens[q], head_dim] of one head, in 64 bits."""
        n = self.lens[q]
        pages = self.table[q][:self.npg(n)]
        d = self.kv.shape[-1]
        return self.by_token()[pool][pages][:, :, head].reshape(-1, d)[:n].double()


def attention(model, layer, q, k, v, seqs, mask=None, nodes=None, scale=None):
    """The definition in 64 bits: (out, lse, A, S, V), where A = sum_j w_j |v_j| by
    element, S the largest sum of |q| |k| scale of a row and V its largest |v| are
    what the error bounds of the tests need."""
    b, t, hq, d = q.shape
    hk = k.shape[2]
    g = hq // hk
    scale = 1 / np.sqrt(d) if scale is None else scale
    out = torch.zeros(b, t, hq, d, dtype=torch.float64)
    lse = torch.full((b, t, hq), -np.inf, dtype=torch.float64)
    a, s, big = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    for i in range(b):
        row = int(seqs[i])
        if not 0 <= row < model.S:
            continue
        count = t if nodes is None else min(max(int(nodes[i]), 0), t)
        for h in range(hk):
            ck, cv = model.context(2 * layer, row, h), model.context(2 * layer + 1, row, h)
            for x in range(count):
                if mask is None:
                    sees = [u for u in range(count) if u <= x]
                else:
                    sees = [u for u in range(count) if int(mask[i, x, u // 64]) >> (u % 64) & 1]
                key = torch.cat([ck, k[i, sees, h].double()])
                val = torch.cat([cv, v[i, sees, h].double()])
                if not len(key):
                    continue
                qq = q[i, x, h * g:(h + 1) * g].double()
                y = qq @ key.T * scale
                z = torch.logsumexp(y, 1)
                w = torch.exp(y - z[:, None])
                out[i, x, h * g:(h + 1) * g] = w @ val
                lse[i, x, h * g:(h + 1) * g] = z
                a[i, x, h * g:(h + 1) * g] = w @ val.abs()
                s[i, x, h * g:(h + 1) * g] = (qq.abs() @ key.abs().T * abs(scale)).amax(1)
                big[i, x, h * g:(h + 1) * g] = val.abs().max()
    return out, lse, a, s, big
