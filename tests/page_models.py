"""Plain models of the chunk attention (64 bits) and of the page operators
(numpy), written from the rules of include/kvq.h."""
import numpy as np

DEV_SLOT, DEV_BLOCK, DEV_SEQ = 1, 2, 4
DEV_REF, DEV_FULL = 16, 32

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4,
                 -6], dtype=np.float64)


def _e4m3():
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 127) == 127 else (
            m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


E4M3 = _e4m3()


class Pages:
    """One layer's NVFP4 cache as bytes [num_blocks, 2, side bytes]."""

    def __init__(self, num_blocks, block, heads, head_size=128, nhd=False,
                 swz_k=False):
        self.nb, self.B, self.H, self.D = num_blocks, block, heads, head_size
        self.S = head_size // 16
        self.nhd, self.swz_k = nhd, swz_k
        self.side = heads * block * (head_size // 2 + self.S)
        self.data = np.zeros((num_blocks, 2, self.side), dtype=np.uint8)

    def places(self, side, off):
        """(data places [H, D/2], scale places [H, S]) of a token."""
        H, B, S, R = self.H, self.B, self.S, self.D // 2
        h = np.arange(H)[:, None]
        c, j = np.arange(R)[None], np.arange(S)[None]
        swz = side == 1 or self.swz_k
        row = (off // 4) * 4 + j // (S // 4) if swz else off + 0 * j
        col = (j % (S // 4)) * 4 + off % 4 if swz else j
        if self.nhd:
            d, s = off * H * R + h * R + c, row * H * S + h * S + col
        else:
            d, s = h * B * R + off * R + c, h * B * S + row * S + col
        return d, H * B * R + s

    def token(self, side, page, off):
        """Dequantised row [H, D] without the tensor scale."""
        d, s = self.places(side, off)
        p = self.data[page, side]
        q = np.stack([E2M1[p[d] & 15], E2M1[p[d] >> 4]], -1)
        q = q.reshape(self.H, self.S, 16) * E4M3[p[s]][..., None]
        return q.reshape(self.H, self.D)

    def rows(self, side):
        """Every token's row: [num_blocks, B, H, D]."""
        out = np.empty((self.nb, self.B, self.H, self.D))
        for off in range(self.B):
            d, s = self.places(side, off)
            p = self.data[:, side]
            q = np.stack([E2M1[p[:, d] & 15], E2M1[p[:, d] >> 4]], -1)
            q = q.reshape(self.nb, self.H, self.S, 16)
            out[:, off] = (q * E4M3[p[:, s]][..., None]).reshape(
                self.nb, self.H, self.D)
        return out

    def fill(self, rng, scale_lo=40, scale_hi=72):
        """Random codes and finite, non-negative scales."""
        cut = self.H * self.B * self.D // 2
        self.data[:, :, :cut] = rng.integers(
            0, 256, self.data[:, :, :cut].shape, dtype=np.uint8)
        self.data[:, :, cut:] = rng.integers(
            scale_lo, scale_hi, self.data[:, :, cut:].shape, dtype=np.uint8)
        return self

    def set_scale(self, side, page, off, head, group, code):
        _, s = self.places(side, off)
        self.data[page, side, s[head, group]] = code


def chunk_attention(pages, q, table, cu, lens, ks, vs, scale):
    """(out, mag, seen, vmax): the attention in 64 bits; mag = sum of weight
    times |V|, seen = tokens a row sees (-1: a row of no sequence)."""
    K, V = pages.rows(0) * ks, pages.rows(1) * vs
    total, hq, D = q.shape
    G = hq // pages.H
    out = np.zeros((total, hq, D))
    mag = np.zeros_like(out)
    seen = np.full(total, -1)
    vmax = np.zeros(total)
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], int(lens[b])
        t = np.arange(L)
        blk = table[b, t // pages.B] if L else np.zeros(0, dtype=int)
        ok = (blk >= 0) & (blk < pages.nb)
        blk = np.where(ok, blk, 0)
        k, v = K[blk, t % pages.B], V[blk, t % pages.B]    # [L, H, D]
        for i in range(n):
            P = L - n + i
            r = cu[b] + i
            see = ok & (t <= P)
            seen[r] = see.sum()
            if not see.any():
                continue
            vmax[r] = np.nanmax(np.abs(v[see]))
            for h in range(hq):
                x = (k[see, h // G] @ q[r, h]) * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[r, h] = w @ v[see, h // G]
                mag[r, h] = w @ np.abs(v[see, h // G])
    return out, mag, seen, vmax


class Pool:
    """The page pool's state and its calls; each returns the error bits."""

    def __init__(self, num_blocks, rows, width, block):
        self.nb, self.B = num_blocks, block
        self.ref = np.zeros(num_blocks, dtype=np.int32)
        self.table = np.full((rows, width), -1, dtype=np.int32)
        self.lens = np.zeros(rows, dtype=np.int32)

    def _page(self, p):
        return 0 <= p < self.nb

    def _pages_for(self, n):
        return -(-n // self.B)

    def _offsets(self, cu, total):
        return (cu[0] == 0 and all(a <= b for a, b in zip(cu, cu[1:]))
                and all(c <= total for c in cu))

    def _take(self, needs):
        """Pages for a list of needs (None: refused before): lists or None."""
        free = np.nonzero(self.ref == 0)[0]
        out, at = [], 0
        for n in needs:
            if n is None:
                out.append(None)
                continue
            ok = n == 0 or at + n <= len(free)
            out.append([int(p) for p in free[at:at + n]] if ok else None)
            at += n
        return out

    def extend(self, ids, cu, total):
        R, W = self.table.shape
        slots = np.full(total, -1, dtype=np.int64)
        if not self._offsets(cu, total):
            bits = DEV_SEQ
            return slots, bits
        bits, needs = 0, []
        for i, s in enumerate(ids):
            add = cu[i + 1] - cu[i]
            n = None
            if not 0 <= s < R or list(ids).count(s) > 1:
                bits |= DEV_SEQ
            else:
                L = int(self.lens[s])
                if L < 0 or L + add > W * self.B:
                    bits |= DEV_SEQ
                elif add and L % self.B and not self._page(
                        self.table[s, L // self.B]):
                    bits |= DEV_BLOCK
                elif add and L % self.B and self.ref[
                        self.table[s, L // self.B]] != 1:
                    bits |= DEV_REF
                else:
                    n = self._pages_for(L + add) - self._pages_for(L)
            needs.append(n)
        for i, (n, got) in enumerate(zip(needs, self._take(needs))):
            if n is None:
                continue
            if got is None:
                bits |= DEV_FULL
                continue
            s = ids[i]
            L, add = int(self.lens[s]), cu[i + 1] - cu[i]
            for j, p in enumerate(got):
                self.table[s, self._pages_for(L) + j] = p
                self.ref[p] = 1
            for k in range(add):
                slots[cu[i] + k] = (int(self.table[s, (L + k) // self.B])
                                    * self.B + (L + k) % self.B)
            self.lens[s] = L + add
        return slots, bits

    def fork(self, parents, children):
        R, W = self.table.shape
        n = len(parents)
        src = np.full(n, -1, dtype=np.int32)
        dst = np.full(n, -1, dtype=np.int32)
        bits, needs = 0, []
        lens = self.lens.copy()
        for p, c in zip(parents, children):
            need = None
            if (not 0 <= p < R or not 0 <= c < R
                    or list(children).count(c) > 1 or lens[c] != 0
                    or (W and self.table[c, 0] >= 0)
                    or not 0 <= lens[p] <= W * self.B):
                bits |= DEV_SEQ
            else:
                need = int(lens[p] % self.B != 0)
                if need and not self._page(self.table[p, lens[p] // self.B]):
                    need = None
                    bits |= DEV_BLOCK
            needs.append(need)
        for i, (need, got) in enumerate(zip(needs, self._take(needs))):
            if need is None:
                continue
            if got is None:
                bits |= DEV_FULL
                continue
            p, c = parents[i], children[i]
            for j in range(lens[p] // self.B):
                page = int(self.table[p, j])
                if self._page(page):
                    self.ref[page] += 1
                else:
                    bits |= DEV_BLOCK
                    page = -1
                self.table[c, j] = page
            if need:
                src[i] = self.table[p, lens[p] // self.B]
                dst[i] = got[0]
                self.table[c, lens[p] // self.B] = got[0]
                self.ref[got[0]] = 1
            self.lens[c] = lens[p]
        return src, dst, bits

    def _drop(self, page):
        if not self._page(page):
            return DEV_BLOCK
        if self.ref[page] <= 0:
            return DEV_REF
        self.ref[page] -= 1
        return 0

    def compact(self, ids, keep, cu, total):
        R, W = self.table.shape
        src = np.full(total, -1, dtype=np.int64)
        dst = np.full(total, -1, dtype=np.int64)
        if not self._offsets(cu, total):
            return src, dst, DEV_SEQ
        bits, plans = 0, []
        for i, s in enumerate(ids):
            k = [int(x) for x in keep[cu[i]:cu[i + 1]]]
            bad = 0
            if not 0 <= s < R or list(ids).count(s) > 1:
                bad = DEV_SEQ
            else:
                L = int(self.lens[s])
                if not 0 <= L <= W * self.B:
                    bad = DEV_SEQ
                for j, x in enumerate(k):
                    if bad & DEV_SEQ and not 0 <= L <= W * self.B:
                        break
                    if not 0 <= x < L or (j and x <= k[j - 1]):
                        bad |= DEV_SEQ
                        continue
                    if not self._page(self.table[s, x // self.B]):
                        bad |= DEV_BLOCK
                    if x != j:
                        to = self.table[s, j // self.B]
                        if not self._page(to):
                            bad |= DEV_BLOCK
                        elif self.ref[to] != 1:
                            bad |= DEV_REF
            bits |= bad
            plans.append(None if bad else k)
        for i, k in enumerate(plans):
            if k is None:
                continue
            s = ids[i]
            for j, x in enumerate(k):
                src[cu[i] + j] = (int(self.table[s, x // self.B]) * self.B
                                  + x % self.B)
                dst[cu[i] + j] = (int(self.table[s, j // self.B]) * self.B
                                  + j % self.B)
        for i, k in enumerate(plans):
            if k is None:
                continue
            s = ids[i]
            self.lens[s] = len(k)
            for j in range(self._pages_for(len(k)), W):
                page = int(self.table[s, j])
                if page >= 0:
                    self.table[s, j] = -1
                    bits |= self._drop(page)
        return src, dst, bits

    def free(self, ids):
        R, W = self.table.shape
        bits = 0
        for s in ids:
            if not 0 <= s < R:
                bits |= DEV_SEQ
                continue
            for j in range(W):
                page = int(self.table[s, j])
                if page >= 0:
                    self.table[s, j] = -1
                    bits |= self._drop(page)
            self.lens[s] = 0
        return bits


def copy_pages(data, src, dst):
    """data [num_blocks, ...] (one cache); returns (bytes after, bits)."""
    out, bits = data.copy(), 0
    for s, d in zip(src, dst):
        if s < 0 or d < 0 or s == d:
            continue
        if s >= len(data) or d >= len(data):
            bits |= DEV_BLOCK
            continue
        out[d] = data[s]
    return out, bits


def move_tokens(pages, src, dst):
    """A Pages' bytes after moves that read everything first; bits."""
    out, bits = pages.data.copy(), 0
    for s, d in zip(src, dst):
        if s < 0 or d < 0 or s == d:
            continue
        if max(s, d) >= pages.nb * pages.B:
            bits |= DEV_SLOT
            continue
        for side in range(2):
            a = np.concatenate([x.ravel() for x in
                                pages.places(side, int(s % pages.B))])
            b = np.concatenate([x.ravel() for x in
                                pages.places(side, int(d % pages.B))])
            out[d // pages.B, side, b] = pages.data[s // pages.B, side, a]
    return out, bits
