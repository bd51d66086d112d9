"""Plain implementations, in fp64 and Python integers, of the operators that
continue one prompt in several ways: attention over a shared prefix, references
to pages, beam search's selection."""
import math

import numpy as np

import decode_reference as ref


class Joined(ref.RefCache):
    """A cache whose requests hold a prefix's slots and then their own: a table row is
    (prefix row, prefix length, own row)."""

    def rows(self, table_row, slots, h):
        before, n, own = table_row
        total = len(slots)
        return np.concatenate([super().rows(before, range(min(n, total)), h),
                               super().rows(own, range(max(0, total - n)), h)])


def shared_attend(q, kc, vc, prefix_table, prefix_lens, groups, table, lens, cu, scale):
    """As decode_reference.attend, over prefix and own slots."""
    rows, total = [], []
    for p in range(len(prefix_lens)):
        for r in range(groups[p], groups[p + 1]):
            rows.append((prefix_table[p], prefix_lens[p], table[r]))
            total.append(prefix_lens[p] + lens[r])
    return ref.attend(q, kc, vc, rows, total, cu, scale)


class Pages:
    """References, and page contents as one list of values for each cache."""

    def __init__(self, refs, block_size, contents=()):
        self.refs, self.bs = [int(x) for x in refs], block_size
        self.contents = [list(c) for c in contents]

    def fork(self, table, lens, parents):
        new, out = [], []
        for p in parents:
            held = -(-lens[p] // self.bs) if p >= 0 else 0
            row = [table[p][i] if i < held else -1 for i in range(len(table[0]) if table else 0)]
            new.append(row)
            out.append(lens[p] if p >= 0 else 0)
        for rows, by in ((new, 1), (table, -1)):
            for row in rows:
                for page in row:
                    if page >= 0:
                        self.refs[page] += by
        return new, out

    def free(self, table):
        for row in table:
            for i, page in enumerate(row):
                if page >= 0:
                    self.refs[page] -= 1
                row[i] = -1

    def reserve(self, table, lens, add):
        """Copies, or None where pages are missing (nothing has changed)."""
        refs, new = list(self.refs), [list(r) for r in table]
        free = [b for b, n in enumerate(refs) if n == 0]
        copies = []
        for row, n, more in zip(new, lens, add):
            copies.append((-1, -1))
            if more == 0:
                continue
            for b in range(n // self.bs, (n + more - 1) // self.bs + 1):
                page = row[b]
                if page >= 0 and refs[page] == 1:
                    continue
                if not free:
                    return None
                row[b] = free.pop(0)
                refs[row[b]] = 1
                if page >= 0:
                    refs[page] -= 1
                    if b == n // self.bs and n % self.bs:
                        copies[-1] = (page, row[b])
        self.refs = refs
        for row, was in zip(new, table):
            was[:] = row
        self.copy(copies)
        return copies

    def copy(self, pairs):
        for c in self.contents:
            for a, b in pairs:
                if a >= 0 and b >= 0:
                    c[b] = c[a]

    def compact(self, tables):
        """Pages held, and each page's new number."""
        held = [n != 0 for n in self.refs]
        used = sum(held)
        moved = [b if h else -1 for b, h in enumerate(held)]
        pairs = list(zip([b for b in range(used, len(held)) if held[b]],
                         [b for b in range(used) if not held[b]]))
        for a, b in pairs:
            moved[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.copy(pairs)
        for table in tables:
            for row in table:
                row[:] = [moved[x] if x >= 0 else x for x in row]
        return used, moved


def beam(logits, scores, done, n, eos):
    """tokens, parents (within the request), scores in fp64, of one request."""
    cand = []
    for k, row in enumerate(logits):
        if not math.isfinite(scores[k]):
            continue
        if done is not None and done[k]:
            cand.append((-float(scores[k]), k, eos))
            continue
        x = np.where(np.isfinite(row), row, -np.inf)
        top = x.max()
        if top == -np.inf:
            continue
        lse = top + math.log(np.exp(x - top).sum())
        # the row's n largest are enough: a stable order by falling logit
        for v in np.argsort(-x, kind="stable")[:n]:
            if x[v] > -np.inf:
                cand.append((-(float(scores[k]) + (x[v] - lse)), k, int(v)))
    cand = sorted(cand)[:n]
    return [c[2] for c in cand], [c[1] for c in cand], [-c[0] for c in cand]
