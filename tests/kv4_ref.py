"""Plain 64-bit model of the paged 4-bit key/value cache on the CPU: the
codec code by code, the page calls entry by entry, attention row by row."""
import numpy as np

BLOCK, GROUP, LIMIT = 128, 32, 26880.0
BAD_INDEX, NO_PAGES, CLAMPED, SHARED = 0x1, 0x4, 0x8, 0x10


def scale_of(code):
    code = np.asarray(code, dtype=np.float64)
    e = np.floor(code / 8)
    return (1 + (code - 8 * e) / 8) * np.exp2(e - 20)


def quantise(x):
    """x [..., D] -> codes [..., D], scale codes [..., D / 32], clamped flag."""
    x = np.asarray(x, dtype=np.float64)
    clamped = bool((~(np.abs(x) <= LIMIT)).any())
    x = np.clip(np.nan_to_num(x, nan=0.0, posinf=LIMIT, neginf=-LIMIT), -LIMIT, LIMIT)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    m, e = np.frexp(np.abs(g).max(-1) / 7.0)
    code = np.where(m > 0, (e - 1 + 20) * 8 + np.rint(m * 16) - 8, 0)
    code = np.clip(code, 0, 255)
    n = np.clip(np.rint(g / scale_of(code)[..., None]), -7, 7)
    return (n + 8).astype(np.int64).reshape(x.shape), code.astype(np.uint8), clamped


def _nibbles(m):
    """Of each of m elements in a row: its byte, and its nibble there."""
    e = np.arange(m)
    nib = (e % 2) * 4 + (e % 8) // 2
    return (e // 8) * 4 + nib // 2, nib % 2


def pack(codes):
    m = codes.shape[-1]
    byte, high = _nibbles(m)
    out = np.zeros(codes.shape[:-1] + (m // 2,), dtype=np.int64)
    for e in range(m):
        out[..., byte[e]] |= codes[..., e] << (4 * high[e])
    return out.astype(np.uint8)


def unpack(b):
    byte, high = _nibbles(2 * b.shape[-1])
    return ((b[..., byte].astype(np.int64) >> (4 * high)) & 15)


class Ref:
    def __init__(self, pages, refs, table, lens, D):
        self.pages, self.refs, self.table, self.lens = (np.array(a) for a in
                                                        (pages, refs, table, lens))
        self.D = D
        self.H = self.pages.shape[1]
        self.status = 0

    # ------------------------------------------------------------- pages
    def count(self, s):
        return -(-int(self.lens[s]) // BLOCK)

    def _ok_slots(self, seqs, n):
        seqs = list(range(n)) if seqs is None else [int(s) for s in seqs]
        return seqs, [0 <= s < len(self.lens) and s not in seqs[:i] for i, s in enumerate(seqs)]

    def resize(self, new, seqs=None):
        seqs, ok = self._ok_slots(seqs, len(new))
        self._take(seqs, ok, [int(x) for x in new], None)

    def _take(self, seqs, ok, new, src):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        at, refs0, copies = 0, self.refs.copy(), []
        for i, s in enumerate(seqs):
            if not ok[i] or not 0 <= new[i] <= self.table.shape[1] * BLOCK:
                self.status |= BAD_INDEX
                continue
            old, had, have = int(self.lens[s]), self.count(s), -(-new[i] // BLOCK)
            if new[i] > old:
                begin = had
                if old % BLOCK and refs0[self.table[s, had - 1]] > 1:
                    begin -= 1
                need = have - begin
                if at + need > len(free) and need:
                    self.status |= NO_PAGES
                    at += need
                    continue
                for j in range(begin, have):
                    p = free[at + j - begin]
                    was = self.table[src[i], j] if src else self.table[s, j] if j < had else -1
                    if was >= 0:
                        copies.append((was, p))
                        if not src:
                            self.refs[was] -= 1
                    self.table[s, j] = p
                    self.refs[p] = 1
                at += need
            else:
                for j in range(have, had):
                    self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1
            self.lens[s] = new[i]
        before = self.pages.copy()
        for a, b in copies:
            self.pages[b] = before[a]

    def fork(self, src, dst, lens=None, deep=False):
        n_seqs = len(self.lens)
        src, dst = [int(x) for x in src], [int(x) for x in dst]
        ok, new = [], []
        for i in range(len(src)):
            good = (0 <= src[i] < n_seqs and 0 <= dst[i] < n_seqs and dst[i] not in dst[:i]
                    and src[i] not in dst and self.lens[dst[i]] == 0)
            L = 0
            if good:
                L = int(self.lens[src[i]]) if lens is None else int(lens[i])
                good = 0 <= L <= self.lens[src[i]]
            ok.append(good)
            new.append(L)
        if deep:
            return self._take(dst, ok, new, src)
        for i in range(len(src)):
            if not ok[i]:
                self.status |= BAD_INDEX
                continue
            for j in range(-(-new[i] // BLOCK)):
                self.table[dst[i], j] = self.table[src[i], j]
                self.refs[self.table[src[i], j]] += 1
            self.lens[dst[i]] = new[i]

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in live if p >= n]
        for a, b in zip(movers, holes):
            self.pages[b] = self.pages[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            for s in range(len(self.lens)):
                row = self.table[s, :self.count(s)]
                row[row == a] = b
        return n

    # ------------------------------------------------------------- codec
    def _halves(self, page, h):
        a, b = BLOCK * self.D // 2, BLOCK * self.D // GROUP
        x = self.pages[page, h]
        return (x[:a].reshape(BLOCK, -1), x[a:a + b].reshape(BLOCK, -1),
                x[a + b:2 * a + b].reshape(self.D, -1), x[2 * a + b:].reshape(-1, BLOCK))

    def _range(self, i, T, seqs, starts, counts, write):
        """(slot, start, count) of entry i, or None."""
        all_seqs = list(range(10 ** 6)) if seqs is None else [int(s) for s in seqs]
        s, count = all_seqs[i], T if counts is None else int(counts[i])
        if not 0 <= s < len(self.lens) or not 0 <= count <= T or \
                (write and seqs is not None and s in all_seqs[:i]):
            self.status |= BAD_INDEX
            return None
        start = int(starts[i]) if starts is not None else int(self.lens[s]) - count if write else 0
        if start < 0 or start + count > self.lens[s]:
            self.status |= BAD_INDEX
            return None
        return s, start, count

    def write(self, k, v, seqs=None, starts=None, counts=None):
        n, H, T, D = k.shape
        for i in range(n):
            r = self._range(i, T, seqs, starts, counts, True)
            if r is None:
                continue
            s, start, count = r
            for j in sorted({p // BLOCK for p in range(start, start + count)}):
                page = self.table[s, j]
                if self.refs[page] > 1:
                    self.status |= SHARED
                    continue
                pos = np.arange(max(start, j * BLOCK), min(start + count, (j + 1) * BLOCK))
                for h in range(H):
                    kc, ks, vc, vs = self._halves(page, h)
                    c, sc, bad = quantise(k[i, h, pos - start])
                    kc[pos - j * BLOCK], ks[pos - j * BLOCK] = pack(c), sc
                    c, sc, bad2 = quantise(v[i, h, pos - start])
                    codes = unpack(vc)
                    codes[:, pos - j * BLOCK] = c.T
                    vc[:] = pack(codes)
                    vs[:, pos - j * BLOCK] = sc.T
                    if bad or bad2:
                        self.status |= CLAMPED

    def head(self, s, h):
        """Keys and values [len, D] of a sequence and head."""
        k, v = [np.zeros((0, self.D))], [np.zeros((0, self.D))]
        for j in range(self.count(s)):
            kc, ks, vc, vs = self._halves(self.table[s, j], h)
            k.append((unpack(kc) - 8) * scale_of(ks).repeat(GROUP, 1))
            v.append(((unpack(vc) - 8) * scale_of(vs).repeat(GROUP, 0)).T)
        L = int(self.lens[s])
        return np.concatenate(k)[:L], np.concatenate(v)[:L]

    def read(self, T, n, seqs=None, starts=None, counts=None, fill=0.0):
        out = np.full((2, n, self.H, T, self.D), fill)
        for i in range(n):
            r = self._range(i, T, seqs, starts, counts, False)
            if r is None:
                continue
            s, start, count = r
            for h in range(self.H):
                for kv, x in zip(out, self.head(s, h)):
                    kv[i, h, :count] = x[start:start + count]
        return out

    # --------------------------------------------------------- attention
    def attn(self, q, seqs=None, tau=None, causal=False, kv_idx=None, kv_cnt=None):
        """out, lse, and what tolerances need: sum p |v| / sum p, the largest
        sum |tau q k| a visible key of the row has, the largest |tau q k|'s of lse."""
        q = np.asarray(q, dtype=np.float64)
        n, Hq, Lq, D = q.shape
        tau = D ** -0.5 if tau is None else tau
        out, size = np.zeros(q.shape), np.zeros(q.shape)
        lse, terms = np.full((n, Hq, Lq), -np.inf), np.zeros((n, Hq, Lq))
        for i in range(n):
            s = i if seqs is None else int(seqs[i])
            if not 0 <= s < len(self.lens):
                self.status |= BAD_INDEX
                continue
            L = int(self.lens[s])
            for h in range(Hq):
                k, v = self.head(s, h // (Hq // self.H))
                for b in range(-(-Lq // BLOCK)):
                    rows = np.arange(b * BLOCK, min(Lq, (b + 1) * BLOCK))
                    if kv_idx is None:
                        at = np.arange(L)
                    else:
                        cnt = min(max(int(kv_cnt[i, h, b]), 0), kv_idx.shape[-1])
                        blocks = kv_idx[i, h, b, :cnt].astype(np.int64)
                        good = (blocks >= 0) & (blocks < self.count(s))
                        if not good.all():
                            self.status |= BAD_INDEX
                        at = (blocks[good][:, None] * BLOCK + np.arange(BLOCK)).reshape(-1)
                        at = at[at < L]
                    if len(at) == 0:
                        continue
                    x = tau * (q[i, h, rows] @ k[at].T)
                    seen = np.ones(x.shape, bool)
                    if causal:
                        seen = at[None] <= (L - Lq + rows)[:, None]
                        x = np.where(seen, x, -np.inf)
                    any_ = seen.any(1)
                    m = np.where(any_, x.max(1), 0.0)
                    p = np.exp(x - m[:, None])
                    z = np.where(any_, p.sum(1), 1.0)
                    out[i, h, rows] = (p @ v[at]) / z[:, None]
                    size[i, h, rows] = (p @ np.abs(v[at])) / z[:, None]
                    lse[i, h, rows] = np.where(any_, m + np.log(z), -np.inf)
                    terms[i, h, rows] = (np.abs(tau * q[i, h, rows]) @ np.abs(k[at]).T).max(1)
        return out, lse, size, terms
