"""Definitions of the decoding operators in float64 (attention over a paged
cache, the cache's upkeep, guided logits), token by token and page by page.
Test infrastructure only; NumPy, no GPU.
"""
import numpy as np


# ---- attention ---------------------------------------------------------------

def visible(tokens, pos, window, sinks):
    """Tokens of ``tokens`` that a query at position ``pos`` sees."""
    seen = tokens <= pos
    if window > 0:
        seen &= (tokens > pos - window) | (tokens < sinks)
    return seen


def row_tokens(cache, row_table, n, page_size):
    """(token numbers, [tokens, kv_heads, dim]) of the row's tokens that have a page."""
    num_pages = cache.shape[0]
    t = np.arange(n)
    page = row_table[t // page_size]
    there = (page >= 0) & (page < num_pages)
    t = t[there]
    return t, cache[page[there], :, t % page_size]


def attention(q, q_offset, k_cache, v_cache, table, kv_len, scale, window=0, sinks=0, k_scale=None, v_scale=None):
    """(out, lse, weight, bound) of every query row, float64: weight is
    sum_t p_t |v_t| per output and bound the largest scale * sum_i |q_i k_ti|
    per (query, head): what a rounding of p or of the scores can reach."""
    tokens, heads, dim = q.shape
    kvh, ps = k_cache.shape[1], k_cache.shape[2]
    group = heads // kvh
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    lse = np.full((tokens, heads), -np.inf)
    bound = np.zeros((tokens, heads))
    for r in range(table.shape[0]):
        n = int(min(max(kv_len[r], 0), table.shape[1] * ps))
        t, k = row_tokens(k_cache, table[r], n, ps)
        _, v = row_tokens(v_cache, table[r], n, ps)
        a, b = int(q_offset[r]), int(q_offset[r + 1])
        for i in range(a, b):
            seen = visible(t, n - (b - i), window, sinks)
            if not seen.any():
                continue
            for h in range(heads):
                kk = k[seen, h // group] * (1.0 if k_scale is None else k_scale[h // group])
                vv = v[seen, h // group] * (1.0 if v_scale is None else v_scale[h // group])
                s = scale * (kk @ q[i, h])
                top = s.max()
                p = np.exp(s - top)
                lse[i, h] = top + np.log(p.sum())
                p /= p.sum()
                out[i, h] = p @ vv
                weight[i, h] = p @ np.abs(vv)
                bound[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, weight, bound


# ---- the cache -----------------------------------------------------------------

class Pages:
    """Tables and pool of a cache, changed one entry at a time."""

    def __init__(self, pool, table, length, refs, page_size):
        self.pool, self.table = np.array(pool), np.array(table)
        self.length, self.refs = np.array(length), np.array(refs)
        self.ps = page_size

    def _ok(self, row):
        return 0 <= row < self.table.shape[0]

    def _free(self):
        return [int(p) for p in np.flatnonzero(self.refs <= 0)]

    def extend(self, rows, count):
        free, asked, named, granted = self._free(), 0, set(), []
        for row, n in zip(rows, count):
            ok = self._ok(row) and row not in named and n >= 0
            if self._ok(row):
                named.add(row)
            if ok:
                old = int(self.length[row])
                ok = old + n <= self.table.shape[1] * self.ps
            if ok:
                first, last = -(-old // self.ps), -(-(old + n) // self.ps)
                at = asked
                asked += last - first
                ok = last == first or asked <= len(free)
            if ok:
                for k in range(first, last):
                    self.table[row, k] = free[at + k - first]
                    self.refs[free[at + k - first]] = 1
                self.length[row] = old + n
            granted.append(int(ok))
        return np.array(granted, np.int32)

    def fork(self, src, dst):
        free, asked, named, granted = self._free(), 0, set(), []
        table, length = self.table.copy(), self.length.copy()
        for s, d in zip(src, dst):
            ok = self._ok(s) and self._ok(d) and s != d and d not in named
            if self._ok(d):
                named.add(d)
            ok = ok and length[d] == 0 and (table.shape[1] == 0 or table[d, 0] < 0)
            if not ok:
                granted.append(0)
                continue
            n = int(length[s])
            full = n // self.ps
            part = int(table[s, full]) if n % self.ps else -1
            if 0 <= part < len(self.refs):
                at, asked = asked, asked + 1
                if asked > len(free):
                    granted.append(0)
                    continue
            self.table[d] = -1
            for k in range(full):
                p = int(table[s, k])
                if 0 <= p < len(self.refs):
                    self.table[d, k] = p
                    self.refs[p] += 1
            if 0 <= part < len(self.refs):
                self.table[d, full] = free[at]
                self.refs[free[at]] = 1
                self.pool[:, free[at]] = self.pool[:, part]
            self.length[d] = n
            granted.append(1)
        return np.array(granted, np.int32)

    def free(self, rows, window=0, sinks=0):
        for row in rows:
            if not self._ok(row):
                continue
            n = int(self.length[row])
            for k in range(self.table.shape[1]):
                a, b = k * self.ps, (k + 1) * self.ps
                if window > 0 and (a < sinks or b > n - window + 1 or b > n):
                    continue
                p = int(self.table[row, k])
                if p >= 0:
                    self.table[row, k] = -1
                    if p < len(self.refs):
                        self.refs[p] -= 1
            if window == 0:
                self.length[row] = 0

    def compact(self):
        live = [int(p) for p in np.flatnonzero(self.refs > 0)]
        count = len(live)
        holes = [p for p in range(count) if self.refs[p] <= 0]
        new = {p: p for p in live}
        for frm, to in zip([p for p in live if p >= count], holes):
            self.pool[:, to] = self.pool[:, frm]
            new[frm] = to
        refs = np.zeros_like(self.refs)
        for p in live:
            refs[new[p]] = self.refs[p]
        # an entry of a page that nobody counts keeps its number
        self.table = np.array([[new.get(int(p), int(p)) if 0 <= p < len(refs) else -1 for p in r] for r in self.table],
                              self.table.dtype).reshape(self.table.shape)
        self.refs = refs
        return len(holes)


# ---- logits ----------------------------------------------------------------------

def guided_logits(logits, cond_row, uncond_row=None, scale=None, history=None, history_len=None, prompt_len=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, temperature=None, mask=None):
    """(z, reach): the logits in float64 and a bound of the magnitudes that
    the fp32 operations round, both divided by the temperature."""
    n, vocab = len(cond_row), logits.shape[1]
    z, reach = np.zeros((n, vocab)), np.zeros((n, vocab))
    for i in range(n):
        c = logits[cond_row[i]].astype(np.float64)
        x, big = c.copy(), np.abs(c)
        if uncond_row is not None and 0 <= uncond_row[i] < len(logits) and scale[i] != 1:
            u, w = logits[uncond_row[i]].astype(np.float64), float(scale[i])
            with np.errstate(invalid="ignore"):
                x = np.where(u == c, c, u + w * (c - u))
                big = np.abs(u) + abs(w) * (np.abs(c) + np.abs(u))
        if history is not None:
            m = min(max(int(history_len[i]), 0), history.shape[1])
            first = 0 if prompt_len is None else int(prompt_len[i])
            seen, count = np.zeros(vocab, bool), np.zeros(vocab)
            for k in range(m):
                t = int(history[i, k])
                if 0 <= t < vocab:
                    seen[t] = True
                    count[t] += k >= first
            r = 1.0 if repetition is None else float(repetition[i])
            x = np.where(seen, np.where(x > 0, x / r, x * r), x)
            big = np.where(seen, big * max(r, 1 / r), big)
            f = 0.0 if frequency is None else float(frequency[i])
            p = 0.0 if presence is None else float(presence[i])
            x = x - f * count - p * (count > 0)
            big = big + abs(f) * count + abs(p) * (count > 0)
        if bias_ids is not None:
            add = {int(t): float(b) for t, b in zip(bias_ids[i], bias[i]) if 0 <= t < vocab}
            for t, b in add.items():
                x[t] += b
                big[t] += abs(b)
        if temperature is not None:
            x, big = x / float(temperature[i]), big / float(temperature[i])
        if mask is not None:
            bits = (mask[i].view(np.uint32)[np.arange(vocab) // 32] >> (np.arange(vocab) % 32).astype(np.uint32)) & 1
            x = np.where(bits == 1, x, -np.inf)
        z[i], reach[i] = x, big
    return z, reach
