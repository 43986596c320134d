"""A plain model of the cache's page bookkeeping (lists and loops on the host), for the tests of kvq_pages_*."""
import numpy as np

PAGE = 16


def pages(tokens):
    return -(-tokens // PAGE)


class Model:
    """Block table, lengths and page counts, and each pool as arrays indexed by page first."""

    def __init__(self, table, lens, refs, pools=()):
        self.table, self.lens, self.refs = np.array(table), np.array(lens), np.array(refs)
        self.pools = [np.array(p) for p in pools]

    def free(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def _held(self, row, tokens):
        return [int(p) for p in row[:pages(tokens)] if 0 <= p < len(self.refs)]

    def fork(self, src, dst):
        """Returns (copy_src, copy_dst), or None when the free pages do not suffice (nothing is then changed)."""
        table, lens, free = self.table.copy(), self.lens.copy(), self.free()
        rows, cs, cd = [], [], []
        for i, s in enumerate(src):
            row = np.full(self.table.shape[1], -1, self.table.dtype)
            u = pages(lens[s])
            row[:u] = table[s][:u]
            a = b = -1
            if lens[s] % PAGE and 0 <= row[u - 1] < len(self.refs) and not (
                    s in dst and s not in src[:i] and self.refs[row[u - 1]] == 1):
                if not free:
                    return None
                a, b = int(row[u - 1]), free.pop(0)
                row[u - 1] = b
            rows.append(row)
            cs.append(a)
            cd.append(b)
        for i, d in enumerate(dst):
            for p in self._held(rows[i], lens[src[i]]):
                self.refs[p] += 1
            for p in self._held(table[d], lens[d]):
                self.refs[p] -= 1
            self.table[d] = rows[i]
            self.lens[d] = lens[src[i]]
        return cs, cd

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            if s >= 0 and d >= 0:
                for p in self.pools:
                    p[d] = p[s]

    def resize(self, seqs, new_lens):
        free = self.free()
        need = sum(max(0, pages(t) - pages(self.lens[s])) for s, t in zip(seqs, new_lens))
        if need > len(free):
            return False
        for s, t in zip(seqs, new_lens):
            had, want = pages(self.lens[s]), pages(t)
            for c in range(had, want):
                p = free.pop(0)
                self.table[s, c] = p
                self.refs[p] += 1
            for p in self.table[s, want:had]:
                if 0 <= p < len(self.refs):
                    self.refs[p] -= 1
            self.table[s, want:had] = -1
            self.lens[s] = t
        return True

    def compact(self, b, n, kept):
        """Keeps the drafted tokens `kept` (rising numbers) of sequence b's last n; returns the length that remains."""
        base = int(self.lens[b]) - n
        for k, j in enumerate(kept):
            s, d = base + j, base + k
            for p in self.pools:  # [pages][kv][heads][16][...]
                p[self.table[b, d // PAGE], :, :, d % PAGE] = p[self.table[b, s // PAGE], :, :, s % PAGE]
        return base + len(kept)
