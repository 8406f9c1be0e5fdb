"""Plain models in 64 bits of the indexer's scores, the selection of blocks
and the attention over what a mask leaves, from the rules of include/kvq.h."""
import numpy as np

from tests.page_models import E4M3


def e4m3_codes(x):
    """fp32 -> e4m3 codes, round to nearest even, saturating: the nearest of
    the 256 values, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]                       # rising, 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def quantize_q(q, weights, scale):
    """(codes, weights_out) of fp32 arrays, in fp32 steps as the rule has
    them."""
    q = q.astype(np.float32)
    s = np.abs(q).max(-1) / np.float32(448.0)
    y = q / np.where(s > 0, s, np.float32(1.0))[..., None]
    w = (weights.astype(np.float32) * np.float32(scale)) * s
    return e4m3_codes(np.where(s[..., None] > 0, y, np.float32(0.0))), w


def rows_of(cu, lens, total):
    """(sequence, tokens that it sees) of each row, (-1, 0) for none."""
    out = [(-1, 0)] * total
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        for i in range(n):
            out[cu[b] + i] = (b, max(L - n + i + 1, 0))
    return out


def score_blocks(q, w, cache, B, D, table, cu, lens, sel, columns):
    """(scores, tolerance), both [rows, columns]; NaN in rows of no sequence.

    Tolerance: e4m3 products are exact; a sum of D of them is off by at most
    D 2^-23 of the sum of their sizes (D additions that may truncate), each of
    the H products with a weight, their sum and the product with the scale by
    (H + 2) 2^-24 of the sum of sizes."""
    total, H = w.shape
    out = np.full((total, columns), np.nan)
    tol = np.zeros((total, columns))
    qv, nb = E4M3[q], cache.shape[0]
    kv = E4M3[cache[:, :B * D].reshape(nb, B, D)]
    sf = np.ascontiguousarray(cache[:, B * D:B * (D + 4)]).view(
        np.float32).reshape(nb, B).astype(np.float64)
    for r, (b, seen) in enumerate(rows_of(cu, lens, total)):
        if b < 0:
            continue
        out[r] = -np.inf
        t = np.arange(seen)
        blk = table[b, t // B] if seen else np.zeros(0, dtype=int)
        ok = (blk >= 0) & (blk < nb)
        blk = np.where(ok, blk, 0)
        k, c = kv[blk, t % B], sf[blk, t % B]                # [T, D], [T]
        with np.errstate(invalid="ignore"):
            x = qv[r] @ k.T                                  # [H, T]
            x = np.where(x < 0, 0.0, x)
            s = (w[r].astype(np.float64) @ x) * c
            size = np.abs(qv[r]) @ np.abs(k).T
            e = np.abs(c) * (np.abs(w[r].astype(np.float64)) @ (
                D * 2.0 ** -23 * size + (H + 2) * 2.0 ** -24 * x))
        s = np.where(ok & ~np.isnan(s), s, -np.inf)
        for j in range(-(-seen // sel)):
            part = slice(j * sel, min((j + 1) * sel, seen))
            out[r, j] = s[part].max()
            tol[r, j] = np.where(np.isfinite(s[part]), e[part], 0).max()
    return out, tol


def select_blocks(scores, cu, lens, sel, top, first, last):
    total = scores.shape[0]
    out = np.full((total, top), -7, dtype=np.int64)      # -7: not written
    for r, (b, seen) in enumerate(rows_of(cu, lens, total)):
        if b < 0:
            continue
        nb = -(-seen // sel)
        x = scores[r, :nb].astype(np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        order = sorted(range(nb), key=lambda j: (
            not (j < first or j >= nb - last), -x[j], j))
        take = sorted(order[:top])
        out[r] = take + [-1] * (top - len(take))
    return out


def masked_attention(pages, q, table, cu, lens, ks, vs, scale, sees):
    """(out, mag, seen, vmax) as page_models.chunk_attention gives them, for
    rows that see the tokens t of sees(b, i, r, n, L) [L] of truth values."""
    K, V = pages.rows(0) * ks, pages.rows(1) * vs
    total, hq, D = q.shape
    G = hq // pages.H
    out = np.zeros((total, hq, D))
    mag = np.zeros_like(out)
    seen = np.full(total, -1)
    vmax = np.zeros(total)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        t = np.arange(L)
        blk = table[b, t // pages.B] if L else np.zeros(0, dtype=int)
        ok = (blk >= 0) & (blk < pages.nb)
        blk = np.where(ok, blk, 0)
        k, v = K[blk, t % pages.B], V[blk, t % pages.B]    # [L, H, D]
        for i in range(n):
            r = cu[b] + i
            see = ok & sees(b, i, r, n, L)
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


def listed_tokens(selected, sel):
    """sees() of lists of blocks: entries that rise, of blocks that the row
    sees something of."""
    def sees(b, i, r, n, L):
        end, out, most = L - n + i + 1, np.zeros(L, dtype=bool), -1
        for e in map(int, selected[r]):
            if 0 <= e and e * sel < end:
                if e > most:
                    out[e * sel:min((e + 1) * sel, end)] = True
                most = max(most, e)
        return out
    return sees


def tree_tokens(mask):
    """sees() of rows of mask words (any integer type)."""
    words = mask.shape[1]

    def sees(b, i, r, n, L):
        out = np.zeros(L, dtype=bool)
        out[:max(L - n, 0)] = True
        for j in range(max(n - L, 0), min(n, 32 * words)):
            out[L - n + j] = (int(mask[r, j // 32]) >> (j % 32)) & 1
        return out
    return sees
