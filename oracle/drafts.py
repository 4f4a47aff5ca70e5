"""Plain CPU definitions of a serving step with drafted tokens (test
infrastructure): rotation and head norm, masks and positions of trees,
verification, and the cache's clean-up. Formats as in ``oracle.fp8``."""

import numpy as np

from oracle.fp8 import E4M3_MAX, e4m3_decode, e4m3_encode, page_scale


def rotate_ref(x, positions, cos_sin, weight=None, eps=1e-6, interleaved=False):
    """x [T, heads, D] -> float32, normed per head and rotated; every product and
    sum rounded by itself. Positions outside the table give NaN."""
    x = np.asarray(x, np.float32)
    rot, half = cos_sin.shape[1], cos_sin.shape[1] // 2
    if weight is not None:
        ms = np.sum(x.astype(np.float64) ** 2, axis=-1, keepdims=True) / x.shape[-1]
        r = (1.0 / np.sqrt(ms + eps)).astype(np.float32)
        x = (x * r) * np.asarray(weight, np.float32)
    known = (positions >= 0) & (positions < len(cos_sin))
    cs = np.where(known[:, None], cos_sin[np.where(known, positions, 0)], np.float32(np.nan)).astype(np.float32)
    c, s = cs[:, None, :half], cs[:, None, half:]
    out = x.copy()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    a, b = x[..., at[0]], x[..., at[1]]
    out[..., at[0]] = a * c - b * s
    out[..., at[1]] = b * c + a * s
    return out


def tree_ref(parents, cu, lens, width):
    """(words int32 [T, width], positions int32 [T]); rows of no sequence are 0."""
    words = np.zeros((len(parents), width), np.uint32)
    pos = np.zeros(len(parents), np.int32)
    for b in range(len(lens)):
        first, n = int(cu[b]), int(cu[b + 1] - cu[b])
        for j in range(n):
            at, depth = j, -1
            while True:
                words[first + j, at // 32] |= np.uint32(1 << (at % 32))
                depth += 1
                up = int(parents[first + at])
                if not 0 <= up < at:
                    break
                at = up
            pos[first + j] = int(lens[b]) - n + depth
    return words.view(np.int32), pos


def verify_ref(probs, tokens, uniform, cu, width, parents=None, draft=None):
    """(kept [B], path [B, width], next [B]) by the rules, in float64."""
    B, V = len(cu) - 1, probs.shape[1]
    kept, path, nxt = np.zeros(B, np.int32), np.full((B, width), -1, np.int32), np.full(B, -1, np.int32)

    def mass(row):
        row = row.astype(np.float64)
        return np.where(row > 0, row, 0.0)  # (NaN too)

    for b in range(B):
        first, n = int(cu[b]), int(cu[b + 1] - cu[b])
        if n <= 0:
            continue
        p = [mass(probs[first + j]) for j in range(n)]
        cur, taken, gone, left = 0, [0], [], 1.0
        for j in range(1, n):
            up = j - 1 if parents is None else int(parents[first + j])
            if up != cur:
                continue
            x = int(tokens[first + j])
            px = p[cur][x] if 0 <= x < V and x not in gone else 0.0
            odds = max(left, 0.0) if draft is None else (mass(draft[first + cur])[x] if 0 <= x < V else 1.0)
            if float(uniform[first + j]) * odds < px:
                cur, gone, left = j, [], 1.0
                taken.append(j)
            else:
                gone.append(x)
                left -= px
        r = p[cur].copy()
        if draft is not None and gone:
            r = np.maximum(r - mass(draft[first + cur]), 0.0)
        elif gone:
            r[[x for x in gone if 0 <= x < V]] = 0.0
        if not r.sum() > 0:
            r = p[cur]
        kept[b] = len(taken)
        path[b, :len(taken)] = taken
        if r.sum() > 0:
            cum = np.cumsum(r)
            past = np.flatnonzero((cum > float(uniform[first]) * cum[-1]) & (r > 0))
            nxt[b] = past[0] if past.size else np.flatnonzero(r > 0)[-1]
    return kept, path, nxt


def keep_ref(k_cache, v_cache, k_scales, v_scales, table, cu, lens, path, kept):
    """The caches [layers, ...] after the kept tokens moved (copies)."""
    kc, vc, ks, vs = k_cache.copy(), v_cache.copy(), k_scales.copy(), v_scales.copy()
    layers, P, H, page, _ = kc.shape

    def at(b, pos):
        slot = pos // page
        p = int(table[b, slot]) if slot < table.shape[1] else -1
        return p if 0 <= p < P else -1

    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        m = min(int(kept[b]), n, path.shape[1])
        if n <= 0 or start < 0:
            continue
        good = [i for i in range(m) if not i <= path[b, i] < n]
        m = good[0] if good else m
        moves = {}  # page -> [(token of the page, source page, its token)]
        for i in range(max(m, 0)):
            to, src = start + i, start + int(path[b, i])
            if to != src and at(b, to) >= 0 and at(b, src) >= 0:
                moves.setdefault(at(b, to), []).append((to % page, at(b, src), src % page))
        for p, move in moves.items():  # (pages in order)
            for c, s, tr in ((kc, ks, False), (vc, vs, True)):
                for layer in range(layers):
                    for h in range(H):
                        tile = c[layer, p, h].T if tr else c[layer, p, h]
                        codes = [(c[layer, q, h].T if tr else c[layer, q, h])[t].copy() for _, q, t in move]
                        from_s = [np.float32(s[layer, q, h]) for _, q, _ in move]
                        codes = [x if np.isfinite(f) else np.full_like(x, 0x7F) for x, f in zip(codes, from_s)]
                        from_s = [f if np.isfinite(f) else np.float32(1) for f in from_s]
                        amax = max(np.max(np.where((x & 0x7F) == 0x7F, 0.0, np.abs(np.nan_to_num(e4m3_decode(x))))) * float(f)
                                   for x, f in zip(codes, from_s))
                        old = np.float32(s[layer, p, h])
                        new = max(old, page_scale(amax)) if amax > 0 else old

                        def over(x, ratio):
                            nan = (x & 0x7F) == 0x7F
                            v = np.clip(e4m3_decode(np.where(nan, 0, x)) * np.float64(np.float32(ratio)), -E4M3_MAX, E4M3_MAX)
                            return np.where(nan, x, e4m3_encode(v))

                        if new != old:
                            tile[:] = over(tile.copy(), old / new)
                        for (t, _, _), x, f in zip(move, codes, from_s):
                            tile[t] = over(x, f / new)
                        s[layer, p, h] = new
    return kc, vc, ks, vs
