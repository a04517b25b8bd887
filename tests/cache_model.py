"""Plain models of the cache-side operators in numpy, 64 bits where numbers are computed. They
share no code with the library; integers and moved bytes are expected to be equal."""
import numpy as np

PAGE = 16


class PoolModel:
    """Page tables, reference counts, lengths and the pool's K and V rows."""

    def __init__(self, table, refs, seq_len, k, v, capacity):
        self.table, self.refs, self.seq_len = table.copy(), refs.copy(), seq_len.copy()
        self.k, self.v, self.capacity = k.copy(), v.copy(), capacity
        self.err = 0

    def active(self, mask):
        return [b for b in range(len(self.seq_len)) if mask is None or mask[b]]

    def reserve(self, n_new=None, mask=None):
        batch = len(self.seq_len)
        ok, wants, spans = [0] * batch, {}, {}
        for b in self.active(mask):
            n = 1 if n_new is None else int(n_new[b])
            length = int(self.seq_len[b])
            if n <= 0:
                ok[b] = 1
                continue
            if length + n > self.capacity:
                self.err |= 0x2
                continue
            if length % PAGE and self.table[b, length // PAGE] < 0:
                self.err |= 0x1
                continue
            spans[b] = range(length // PAGE, (length + n - 1) // PAGE + 1)
        leans = {}                      # the last sequence that leaves a page to this one
        for b in spans:
            wants[b] = []
            for c in spans[b]:
                e = self.table[b, c]
                before = [o for o in spans if o < b and c in spans[o] and self.table[o, c] == e]
                if e < 0 or (self.refs[e] > 1 and self.refs[e] - len(before) > 1):
                    wants[b].append(c)
                elif before and self.refs[e] > 1:
                    leans.setdefault(b, set()).update(before)
        free = [int(i) for i in np.flatnonzero(self.refs == 0)]
        used = 0
        for b in spans:
            used += len(wants[b])
            if (wants[b] and used > len(free)) or any(not ok[o] for o in leans.get(b, ())):
                self.err |= 0x10
                continue
            ok[b] = 1
            for c, new in zip(wants[b], free[used - len(wants[b]):used]):
                old, rows = self.table[b, c], int(self.seq_len[b]) % PAGE
                self.table[b, c] = new
                self.refs[new] = 1
                if old >= 0:
                    self.refs[old] -= 1
                    if c == spans[b][0] and rows:
                        for t in (self.k, self.v):
                            t[:, new, :, :rows] = t[:, old, :, :rows]
        return np.array(ok, np.uint8)

    def _drop(self, b, cols):
        for c in cols:
            if self.table[b, c] >= 0:
                self.refs[self.table[b, c]] -= 1
                self.table[b, c] = -1

    def release(self, mask=None):
        for b in self.active(mask):
            self._drop(b, range(self.table.shape[1]))
            self.seq_len[b] = 0

    def evict(self, n_sink, n_window, mask=None):
        for b in self.active(mask):
            live = set(range(n_sink)) | set(range(max(0, self.seq_len[b] - n_window), self.capacity))
            self._drop(b, [c for c in range(self.table.shape[1])
                           if not live & set(range(c * PAGE, (c + 1) * PAGE))])

    def append(self, k_new, v_new, start, mask=None):
        for b in self.active(mask):
            for i in range(start[b], start[b + 1]):
                p = int(self.seq_len[b]) + i - start[b]
                page = self.table[b, p // PAGE]
                self.k[:, page, :, p % PAGE] = k_new[:, i]
                self.v[:, page, :, p % PAGE] = v_new[:, i]
            self.seq_len[b] += start[b + 1] - start[b]

    def compact(self):
        used = self.refs != 0
        n = int(used.sum())
        to = [i for i in range(n) if not used[i]]
        of = [i for i in range(n, len(used)) if used[i]]
        for a, c in zip(to, of):
            self.k[:, a], self.v[:, a] = self.k[:, c], self.v[:, c]
            self.table[self.table == c] = a
            self.refs[a], self.refs[c] = self.refs[c], 0
        return n

    def reorder(self, src):
        for e in self.table[self.table >= 0]:
            self.refs[e] -= 1
        self.table, self.seq_len = self.table[src], self.seq_len[src]
        for e in self.table[self.table >= 0]:
            self.refs[e] += 1


def window_attention(q, k, v, length, n_sink, n_window):
    """q [m][Hq][D] of the last m positions, k and v [Hkv][length][D] -> float64 [m][Hq][D], and
    the same with |v| (the scale that rounding errors of the weights go by)."""
    m, hq, d = q.shape
    group = hq // k.shape[0]
    pos, j = np.arange(length - m, length)[:, None], np.arange(length)
    seen = (j <= pos) & ((j < n_sink) | (j > pos - n_window))
    used = seen.any(0)
    out, mag = np.zeros(q.shape, np.float64), np.zeros(q.shape, np.float64)
    for h in range(hq):
        kh, vh = k[h // group][used].astype(np.float64), v[h // group][used].astype(np.float64)
        z = np.where(seen[:, used], q[:, h].astype(np.float64) @ kh.T / np.sqrt(d), -np.inf)
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[:, h], mag[:, h] = w @ vh, w @ np.abs(vh)
    return out, mag


def beam_select(x, cum, done, scale, eos, n_beams):
    """x [groups * n_beams][vocab]; returns parent, token, cum, done of the kept candidates."""
    rows, vocab = x.shape
    parent, token, score, fin = [], [], [], []
    with np.errstate(all="ignore"):
        for g in range(rows // n_beams):
            cand = []
            for r in range(g * n_beams, (g + 1) * n_beams):
                w = 1.0 if scale is None else float(scale[r])
                if done is not None and done[r]:
                    s = float(cum[r]) if np.isfinite(cum[r]) else -np.inf
                    cand.append((-s * w, r, eos, s, 1))
                    continue
                row = x[r].astype(np.float64)
                top = row.max()
                s = float(cum[r]) + (row - top - np.log(np.exp(row - top).sum()))
                s = np.where(np.isfinite(s), s, -np.inf)
                best = np.lexsort((np.arange(vocab), -s))[:n_beams]
                cand += [(-s[t] * w, r, int(t), s[t], int(t == eos)) for t in best]
            for c in sorted(cand)[:n_beams]:
                parent.append(c[1])
                token.append(c[2])
                score.append(c[3])
                fin.append(c[4])
    return np.array(parent), np.array(token), np.array(score), np.array(fin)
