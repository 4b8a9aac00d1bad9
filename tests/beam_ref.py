"""Plain fp64 forms of the beam-search operators on the host, straight from
their definitions, over the automaton's edge list (original state ids)."""
import numpy as np


def edge_tokens(aut):
    """Per state a list of (sorted token array, target)."""
    out = [[] for _ in range(aut.S)]
    for e in range(aut.E):
        lab = aut.edge_label(e)
        if lab.size:
            out[int(aut.src[e])].append((lab, int(aut.dst[e])))
    return out


def select(aut, x, scores, sets, K, mode="logits", reach=None, edges=None):
    """x [B, Kin, V] fp64, scores [B, Kin], sets: [B][Kin] python sets.
    Returns scores [B, K] (fp64), tokens, parents, sets, status [B]."""
    edges = edges or edge_tokens(aut)
    B, Kin, V = x.shape
    sc = np.full((B, K), -np.inf)
    tok = np.full((B, K), -1, np.int64)
    par = np.tile(np.arange(K) % Kin, (B, 1))
    new = [[set() for _ in range(K)] for _ in range(B)]
    status = np.zeros(B, np.int64)
    for b in range(B):
        cand = []
        bad = False
        for k in range(Kin):
            s = float(scores[b, k])
            if np.isnan(s) or s == np.inf:
                bad = True
                continue
            if s == -np.inf:
                continue
            may = np.zeros(V, bool)
            for q in sets[b][k]:
                for lab, to in edges[q]:
                    if reach is None or reach[to]:
                        may[lab] = True
            v = np.flatnonzero(may)
            row = x[b, k]
            if mode == "probs":
                xv = row[v]
                if not (np.isfinite(xv) & (xv >= 0)).all():
                    bad = True
                    continue
                with np.errstate(divide="ignore"):
                    key = s + np.log(xv)
            else:
                if np.isnan(row).any() or (row == np.inf).any():
                    bad = True
                    continue
                m = row.max()
                if m == -np.inf:
                    continue
                key = s + (row[v] - (m + np.log(np.exp(row - m).sum())))
            cand += [(-kk, k * V + int(vv)) for kk, vv in zip(key, v) if kk > -np.inf]
        if bad:
            status[b] = 4
            continue
        cand.sort()
        if not cand:
            status[b] = 1
        for j, (nk, flat) in enumerate(cand[:K]):
            sc[b, j], par[b, j], tok[b, j] = -nk, flat // V, flat % V
            for q in sets[b][flat // V]:
                for lab, to in edges[q]:
                    if (reach is None or reach[to]) and flat % V in lab:
                        new[b][j].add(to)
    return sc, tok, par, new, status


def words_of(sets, W):
    """[B][K] sets of compact ids -> int32 words [B, K, W]."""
    a = np.zeros((len(sets), len(sets[0]), W), np.uint32)
    for b, row in enumerate(sets):
        for k, q in enumerate(row):
            for s in q:
                a[b, k, s // 32] |= np.uint32(1 << (s % 32))
    return a.view(np.int32)


def sets_of(words):
    w = np.asarray(words).view(np.uint32)
    bits = (w[..., None] >> np.arange(32, dtype=np.uint32)) & 1
    flat = bits.reshape(w.shape[0], w.shape[1], -1)
    return [[set(np.flatnonzero(flat[b, k]).tolist()) for k in range(w.shape[1])]
            for b in range(w.shape[0])]


def trace(tokens, parents):
    T, B, K = tokens.shape
    out = np.full((B, K, T), -1, np.int64)
    for b in range(B):
        for k in range(K):
            j = k
            for t in range(T - 1, -1, -1):
                if not 0 <= j < K:
                    break
                out[b, k, t] = tokens[t, b, j]
                j = parents[t, b, j]
    return out


def reorder(x, parents):
    B, K = parents.shape
    p = np.where((parents >= 0) & (parents < K), parents, np.arange(K))
    return x[np.arange(B)[:, None], p]


def search(aut, logits_of, B, L, K, reach, mode="logits"):
    """The whole search with fp32 scores between steps; reach[r] the states r
    tokens before acceptance.  Returns tokens [B, K, L], fp64 scores."""
    edges = edge_tokens(aut)
    scores = np.full((B, K), -np.inf, np.float32)
    scores[:, 0] = 0
    sets = [[{aut.start} if k == 0 else set() for k in range(K)] for _ in range(B)]
    toks = np.zeros((L, B, K), np.int64)
    pars = np.zeros((L, B, K), np.int64)
    for t in range(L):
        x = logits_of(t, toks[:t], pars[:t])
        sc, toks[t], pars[t], sets, status = select(aut, x, scores, sets, K, mode,
                                                    reach[L - t - 1], edges)
        scores = sc.astype(np.float32)
    return trace(toks, pars), scores, status
