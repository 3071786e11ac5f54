"""Plain implementations of the paged-cache operators in 64 bits (no code shared with the library): sequences as lists on the
host, attention and beams in float64."""
import numpy as np
import torch


def pages_of(rows, page):
    return -(-rows // page)


def pool_state(rs, lengths, page, spare=5, width=None):
    """A table of private pages in a random order, lengths and counts."""
    held = [pages_of(n, page) for n in lengths]
    n_pages = sum(held) + spare
    ids = rs.permutation(n_pages)[:sum(held)]
    width = width or max(held) + 2
    table = np.full((len(lengths), width), -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = ids[at:at + h]
        at += h
    return table, np.array(lengths, dtype=np.int32), np.bincount(ids, minlength=n_pages).astype(np.int32)


def fork(table, length, parent, refs, page):
    out = np.full((len(parent), table.shape[1]), -1, dtype=np.int32)
    new, refs = np.zeros(len(parent), dtype=np.int32), refs.copy()
    for r in range(len(table)):
        for p in table[r, :pages_of(length[r], page)]:
            refs[p] -= 1
    for i, up in enumerate(parent):
        if 0 <= up < len(table):
            held = pages_of(length[up], page)
            out[i, :held] = table[up, :held]
            new[i] = length[up]
            for p in table[up, :held]:
                refs[p] += 1
    return out, new, refs


def extend(table, length, refs, counts, page):
    """One sequence after the other; returns table, length, refs, rows, pos, pairs and how many could not be extended."""
    table, length, refs = table.copy(), length.copy(), refs.copy()
    rows, pos, pairs, bad, dry = [], [], [], 0, False
    for s, n in enumerate(counts):
        old, len_s = pages_of(max(length[s], 0), page), int(length[s])
        ok = len_s >= 0 and len_s + n <= table.shape[1] * page
        part = ok and n > 0 and len_s % page != 0
        if part and not 0 <= table[s, old - 1] < len(refs):
            ok = part = False
        cow = bool(part and refs[table[s, old - 1]] > 1)
        want = (pages_of(len_s + n, page) - old if ok else 0) + cow
        free = np.flatnonzero(refs == 0)
        if ok and want > len(free):
            dry = True
        if not ok or dry:
            bad += n > 0
            pairs.append((-1, -1))
            rows += [-1] * n
            pos += list(range(len_s, len_s + n)) if ok else [0] * n
            continue
        take = list(free[:want])
        refs[take] = 1
        if cow:
            was = table[s, old - 1]
            refs[was] -= 1
            pairs.append((was, take[0]))
            table[s, old - 1] = take.pop(0)
        else:
            pairs.append((-1, -1))
        table[s, old:old + len(take)] = take
        length[s] += n
        pos += list(range(len_s, len_s + n))
        rows += [table[s, p // page] * page + p % page for p in range(len_s, len_s + n)]
    return table, length, refs, np.array(rows), np.array(pos), np.array(pairs), bad


def compact(refs, table, length, page):
    used = refs > 0
    count = int(used.sum())
    moves = list(zip(count + np.flatnonzero(used[count:]), np.flatnonzero(~used[:count])))
    refs, table, to = refs.copy(), table.copy(), dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    for s in range(len(table)):
        for p in range(pages_of(length[s], page)):
            table[s, p] = to.get(table[s, p], table[s, p])
    return refs, table, np.array(moves, dtype=np.int32).reshape(-1, 2), count


def rows_of(table, n, page):
    return np.array([table[t // page] * page + t % page for t in range(n)], dtype=np.int64)


def attend(q, k, v, table, counts, length, page, window=0, cap=0.0, slopes=None):
    """(out, sum of |weight| |value|) in float64 on q's device; tokens that see nothing get 0."""
    T, Hq, D = q.shape
    G = Hq // k.shape[0]
    out, size = (torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device) for _ in range(2))
    at = 0
    for s, n in enumerate(counts):
        if n == 0:
            continue
        seen = int(length[s])
        rows = torch.from_numpy(rows_of(table[s], seen, page)).to(q.device)
        pos = (seen - n + torch.arange(n, device=q.device))[:, None]
        key = torch.arange(seen, device=q.device)[None, :]
        see = (key <= pos) & ((key > pos - window) if window else True)
        some = see.any(1)
        for h in range(Hq):
            if seen == 0:
                break
            kk, vv = k[h // G, rows].double(), v[h // G, rows].double()
            x = q[at:at + n, h].double() @ kk.T / D ** 0.5
            if cap:
                x = cap * torch.tanh(x / cap)
            if slopes is not None:
                x = x - slopes[h].double() * (pos - key)
            x = torch.where(see, x, -torch.inf)
            x = torch.where(some[:, None], x, 0.0)
            w = torch.where(see, torch.softmax(x, -1), 0.0)
            # a value is left out of a sum, not multiplied by 0, where it is not seen
            if torch.isfinite(vv).all():
                out[at:at + n, h], size[at:at + n, h] = w @ vv, w @ vv.abs()
            else:
                for i in range(n):
                    out[at + i, h], size[at + i, h] = w[i, see[i]] @ vv[see[i]], w[i, see[i]] @ vv[see[i]].abs()
        at += n
    return out, size


def beam(logits, scores, W, K, done=None, eos=-1, lengths=None, alpha=0.0):
    """parent, token, score, done of every group, in float64 (NumPy)."""
    N, V = logits.shape
    parent, token, score, fin = [], [], [], []
    for g in range(N // W):
        cand = []
        for b in range(g * W, (g + 1) * W):
            s = float(scores[b])
            if not np.isfinite(s):
                continue
            if done is not None and done[b]:
                cand.append((s / max(int(lengths[b]), 1) ** alpha if alpha else s, b, eos, s, 1))
                continue
            x = logits[b].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            m = x.max()
            if not np.isfinite(m):
                continue
            total = s + (x - (m + np.log(np.exp(x - m).sum())))
            rank = total / max(int(lengths[b]) + 1, 1) ** alpha if alpha else total
            for v in np.lexsort((np.arange(V), -rank))[:K]:
                if total[v] > -np.inf:
                    cand.append((rank[v], b, int(v), total[v], int(v == eos)))
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        cand = cand[:K] + [(0, -1, -1, -np.inf, 0)] * (K - len(cand[:K]))
        parent += [c[1] for c in cand]
        token += [c[2] for c in cand]
        score += [c[3] for c in cand]
        fin += [c[4] for c in cand]
    return np.array(parent), np.array(token), np.array(score), np.array(fin)
