"""A page table in plain Python: what the page-table entry points do, one
sequence and one page at a time. The tests hold the kernels to it bit for bit."""
import numpy as np


class PageModel:
    def __init__(self, num_pages, page_size, max_seqs, max_pages):
        self.N, self.P, self.S, self.M = num_pages, page_size, max_seqs, max_pages
        self.lens = [0] * max_seqs
        self.list = [[-1] * max_pages for _ in range(max_seqs)]
        self.rc = [0] * num_pages
        self.free = [num_pages - 1 - i for i in range(num_pages)]   # whole array, stale behind count
        self.count = num_pages

    def pages(self, n):
        return -(-n // self.P)

    def words(self):
        """free_count and the table's words in the buffer's order."""
        body = self.lens + [p for row in self.list for p in row] + self.rc + self.free
        return self.count, np.array(body, dtype=np.int32)

    def _take(self):
        self.count -= 1
        return self.free[self.count]

    def reserve(self, ids, new, pools=()):
        """Slots of the new tokens, or None (nothing changed) where the call has to fail.
        pools: arrays [layers, N, Hkv, P, x], pages copied in place."""
        if len(set(ids)) < len(ids) or any(i < 0 or i >= self.S for i in ids) or min(new, default=0) < 0:
            return None
        if any(self.lens[i] + n > self.M * self.P for i, n in zip(ids, new)):
            return None
        tails = {}
        for at, (i, n) in enumerate(zip(ids, new)):
            L = self.lens[i]
            if n > 0 and L % self.P:
                p = self.list[i][L // self.P]
                if self.rc[p] > 1:
                    tails.setdefault(p, []).append(at)
        cow = set()
        for p, writers in tails.items():
            cow.update(writers[1:] if len(writers) == self.rc[p] else writers)
        need = sum(self.pages(self.lens[i] + n) - self.pages(self.lens[i]) + (at in cow)
                   for at, (i, n) in enumerate(zip(ids, new)))
        if need > self.count:
            return None
        slots, moves = [], []
        for at, (i, n) in enumerate(zip(ids, new)):
            L, row = self.lens[i], self.list[i]
            if at in cow:
                old, page = row[L // self.P], self._take()
                self.rc[old] -= 1
                self.rc[page] = 1
                row[L // self.P] = page
                moves.append((old, page, L % self.P))
            for e in range(self.pages(L), self.pages(L + n)):
                row[e] = self._take()
                self.rc[row[e]] = 1
            slots += [row[(L + t) // self.P] * self.P + (L + t) % self.P for t in range(n)]
            self.lens[i] = L + n
        for pool in pools:
            for old, page, rows in moves:
                pool[:, page, :, :rows] = pool[:, old, :, :rows]
        return slots

    def fork(self, src, dst):
        ok = (len(set(dst)) == len(dst) and all(0 <= i < self.S for i in list(src) + list(dst))
              and not set(src) & set(dst) and all(self.lens[d] == 0 for d in dst))
        if not ok:
            return False
        for s, d in zip(src, dst):
            self.lens[d] = self.lens[s]
            self.list[d] = list(self.list[s])
            for p in self.list[s][:self.pages(self.lens[s])]:
                self.rc[p] += 1
        return True

    def truncate(self, ids, new):
        ok = (len(set(ids)) == len(ids) and all(0 <= i < self.S for i in ids)
              and all(0 <= n <= self.lens[i] for i, n in zip(ids, new)))
        if not ok:
            return False
        entries = []
        for i, n in zip(ids, new):
            for e in range(self.pages(n), self.pages(self.lens[i])):
                entries.append(self.list[i][e])
                self.rc[self.list[i][e]] -= 1
                self.list[i][e] = -1
            self.lens[i] = n
        gone = []
        for p in entries:
            if self.rc[p] == 0 and p not in gone:
                gone.append(p)
        for j, p in enumerate(gone):
            self.free[self.count + len(gone) - 1 - j] = p
        self.count += len(gone)
        return True

    def compact(self, pools=()):
        live = [p for p in range(self.N) if self.rc[p] > 0]
        kept = len(live)
        holes = [p for p in range(kept) if self.rc[p] == 0]
        movers = [p for p in live if p >= kept]
        to = {p: p for p in live}
        to.update(zip(movers, holes))
        for pool in pools:
            for a, b in zip(movers, holes):
                pool[:, b] = pool[:, a]
        rc = [0] * self.N
        for p in live:
            rc[to[p]] = self.rc[p]
        self.rc = rc
        self.list = [[to[p] if p >= 0 else -1 for p in row] for row in self.list]
        for i in range(self.N - kept):
            self.free[i] = self.N - 1 - i
        self.count = self.N - kept
        return [to.get(p, -1) for p in range(self.N)]
