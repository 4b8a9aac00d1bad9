"""What is measured of the beam-search operators: the joint selection of K
beams over beams and vocabulary under a compiled automaton (beam_select), the
reordering of the model's states by the chosen parents (beam_reorder), and the
hypotheses read back from the recorded parents (beam_trace).

``run`` computes a case in plain torch operations, or (``own``) through the
package's entry points.  ``exact`` computes it on the host in 64 bits from the
definition.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "u8": torch.uint8}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "u8": 1}


# ------------------------------------------------------------------- cases
def _select(name, kind, mode, dtype, B, K, V, S, steps, pad=0, fresh=False):
    return {"name": name, "op": "select", "kind": kind, "mode": mode, "dtype": dtype, "B": B,
            "K": K, "V": V, "S": S, "steps": steps, "pad": pad, "fresh": fresh}


def _reorder(name, dtype, B, K, tensors, heads, cap, length, dim, inplace):
    return {"name": name, "op": "reorder", "dtype": dtype, "B": B, "K": K, "tensors": tensors,
            "heads": heads, "cap": cap, "length": length, "dim": dim, "inplace": inplace}


def listed():
    return [
        # one interactive request, four beams, an automaton of a few dozen
        # states over a small vocabulary: the call's latency is all there is
        _select("select-interactive", "json", "logits", "f32", B=1, K=4, V=1024, S=32, steps=64),
        # the first step of a request (only beam 0 is live) on a 32k vocabulary
        _select("select-first-step", "json", "logits", "f16", B=1, K=8, V=32000, S=64, steps=128,
                fresh=True),
        # odd vocabulary and counts, rows of a padded output (odd row pitch)
        _select("select-odd", "json", "logits", "f16", B=3, K=5, V=50257, S=33, steps=37, pad=46),
        # the benchmark's JSON-like automaton: 4 rows, 256 states, 151,936 tokens
        _select("select-json", "json", "logits", "bf16", B=4, K=8, V=151936, S=256, steps=256),
        # K best strings of one denoising step: p itself, one row shared by the beams
        _select("select-probs", "json", "probs", "f32", B=4, K=16, V=151936, S=256, steps=100),
        # range labels (the batch-throughput automaton), many beams, fp32 logits
        _select("select-range", "range", "logits", "f32", B=16, K=32, V=151936, S=1024, steps=512),
        # a nondeterministic automaton: every beam carries a set of states
        _select("select-nfa", "nfa", "logits", "bf16", B=4, K=16, V=32768, S=2000, steps=64),
        # batch serving, no length limit in sight (no lookahead)
        _select("select-batch", "json", "logits", "bf16", B=64, K=16, V=151936, S=256, steps=0),
        # byte caches with odd sizes, into second buffers
        _reorder("reorder-odd", "u8", B=3, K=5, tensors=6, heads=3, cap=1000, length=777, dim=75,
                 inplace=False),
        # batch serving: the keys and values of four layers, in place
        _reorder("reorder-batch", "bf16", B=8, K=8, tensors=8, heads=8, cap=1024, length=1000,
                 dim=128, inplace=True),
        # the hypotheses of one short answer, and of a batch of long ones
        {"name": "trace-short", "op": "trace", "T": 33, "B": 1, "K": 4},
        {"name": "trace-long", "op": "trace", "T": 2048, "B": 64, "K": 16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    u = rng.random()
    if u < 0.6:
        kind = rng.choice(["json", "json", "range", "nfa"])
        mode = "probs" if rng.random() < 0.25 else "logits"
        dtype = "f32" if mode == "probs" else rng.choice(["f32", "f16", "bf16", "bf16"])
        B, K = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        V = min(_log_int(rng, 512, 200000), 120_000_000 // (B * K))
        if kind == "nfa":
            S = _log_int(rng, 64, 2000)
            V = min(V, 40000, 12_000_000 // (B * K))
        else:
            S = _log_int(rng, 16, 1024 if kind == "range" else 256)
        steps = 0 if rng.random() < 0.3 else rng.randint(12, 300)
        c = _select("", kind, mode, dtype, B, K, V, S, steps, pad=rng.choice([0, 0, 1, 5, 64]),
                    fresh=rng.random() < 0.1)
    elif u < 0.85:
        dtype = rng.choice(["f32", "bf16", "bf16", "u8"])
        B, K = _log_int(rng, 1, 16), _log_int(rng, 1, 64)
        heads, dim = rng.randint(1, 8), rng.choice([33, 64, 75, 80, 128, 128])
        tensors = rng.randint(1, 16)
        room = 500_000_000 // (B * K * heads * dim * tensors * SIZE[dtype])
        cap = max(1, min(_log_int(rng, 1, 4096), room))
        c = _reorder("", dtype, B, K, tensors, heads, cap, rng.randint(max(1, cap // 2), cap), dim,
                     rng.random() < 0.6)
    else:
        c = {"op": "trace", "T": _log_int(rng, 1, 2048), "B": _log_int(rng, 1, 64),
             "K": _log_int(rng, 1, 16)}
    c.pop("name", None)
    return c


# --------------------------------------------------------------- automata
def _edges(kind, S, V, seed):
    """(edges, accept): edges as (source, target, sorted tokens or one
    half-open token range)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    edges = []
    if kind == "json":
        # structural states: a few tokens of a common pool, each with its own
        # target; string states: most of the vocabulary leads back, a quote out
        strings = np.zeros(S, bool)
        strings[rng.choice(np.arange(1, S), max(1, S // 10), replace=False)] = True
        structural = np.flatnonzero(~strings)
        pool = rng.choice(V, min(256, V // 2), replace=False)
        for s in range(S):
            if strings[s]:
                inside = rng.random(V) < 0.66
                inside[pool[0]] = False
                edges.append((s, s, np.flatnonzero(inside)))
                edges.append((s, int(rng.choice(structural)), pool[:1]))
            else:
                toks = np.sort(rng.choice(pool, int(rng.integers(1, min(64, pool.size) + 1)),
                                          replace=False))
                to = rng.integers(0, S, toks.size)
                for t in np.unique(to):
                    edges.append((s, int(t), toks[to == t]))
        accept = rng.choice(structural, min(4, structural.size), replace=False)
    elif kind == "range":
        for s in range(S):
            cuts = np.sort(rng.choice(V + 1, 32, replace=False))
            for j, t in enumerate(rng.integers(0, S, 16)):
                edges.append((s, int(t), (int(cuts[2 * j]), int(cuts[2 * j + 1]))))
        accept = rng.choice(S, 4, replace=False)
    else:
        sizes = np.minimum(rng.geometric(1 / 50.0, 10 * S), V)
        for n, a, b in zip(sizes, rng.integers(0, S, 10 * S), rng.integers(0, S, 10 * S)):
            edges.append((int(a), int(b), np.unique(rng.integers(0, V, n))))
        accept = rng.choice(S, 16, replace=False)
    return edges, np.sort(accept).astype(np.int32)


def _reach(edges, accept, S, r):
    """States from which an accepting state is exactly r steps away."""
    src = np.array([e[0] for e in edges])
    dst = np.array([e[1] for e in edges])
    now = np.zeros(S, bool)
    now[accept] = True
    for _ in range(r):
        before, now = now, np.zeros(S, bool)
        now[src[before[dst]]] = True
    return now


def _table(case, edges, accept):
    import constrained_decoding_diffusion_amd as fa
    flags = fa.FA_NO_TRIM | fa.FA_BEAMS | (fa.FA_NFA if case["kind"] == "nfa" else fa.FA_DFA)
    flags |= fa.FA_LABEL_RANGES if case["kind"] == "range" else 0
    labels = [np.asarray(e[2], np.int32) for e in edges]
    off = np.zeros(len(edges) + 1, np.int64)
    np.cumsum([x.size for x in labels], out=off[1:])
    table = fa.Table(case["S"], case["V"], 0, accept, np.array([e[0] for e in edges]),
                     np.array([e[1] for e in edges]), off, np.concatenate(labels), flags)
    return fa, table.upload()


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _select_inputs(case, seed):
    B, K, V, S = case["B"], case["K"], case["V"], case["S"]
    g = _generator(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    edges, accept = _edges(case["kind"], S, V, seed + 1)
    rows = 1 if case["mode"] == "probs" else K
    x = torch.empty((B, rows, V + case["pad"]), dtype=DTYPES[case["dtype"]], device="cuda")
    bias = -1.1 * torch.log(torch.arange(V + case["pad"], device="cuda") + 1.0)
    for b in range(B):
        z = torch.randn((rows, V + case["pad"]), generator=g, device="cuda") * 3 + bias
        if case["mode"] == "probs":
            z = torch.softmax(z[:, :V].double(), -1)
            x[b, :, :V] = z.to(x.dtype)
        else:
            x[b] = z.to(x.dtype)
    x = x[:, :, :V].expand(B, K, V)
    scores = -torch.rand((B, K), generator=g, device="cuda").mul(6).sort(-1).values - 20
    if case["fresh"]:
        scores[:] = -math.inf
        scores[:, 0] = 0
    # the beams' states: half of them where most of the vocabulary is allowed
    loops = np.array([e[0] for e in edges if e[0] == e[1]] or [0])
    ids = np.where(rng.random((B, K)) < 0.5, rng.choice(loops, (B, K)), rng.integers(0, S, (B, K)))
    ids[:, 0] = rng.choice(loops, B)
    sets = np.zeros((B, K, S), bool)
    np.put_along_axis(sets, ids[..., None], True, -1)
    if case["kind"] == "nfa":
        np.put_along_axis(sets, rng.integers(0, S, (B, K, 7)), True, -1)
    return {"logits": x, "scores": scores, "sets": sets, "ids": ids, "edges": edges,
            "accept": accept}


def _words(sets):
    """Bitsets of the last axis in int32 words (bit s % 32 of word s // 32)."""
    S = sets.shape[-1]
    w = torch.nn.functional.pad(sets, (0, -S % 32)).unflatten(-1, (-1, 32)).to(torch.int64)
    return (w << torch.arange(32, device=sets.device)).sum(-1).to(torch.int32)


def _reorder_inputs(case, seed):
    B, K = case["B"], case["K"]
    g = _generator(seed)
    shape = (B, K, case["heads"], case["cap"], case["dim"])
    caches = []
    for _ in range(case["tensors"]):
        if case["dtype"] == "u8":
            caches.append(torch.randint(0, 256, shape, generator=g, device="cuda",
                                        dtype=torch.uint8))
        else:
            caches.append(torch.randn(shape, generator=g, device="cuda",
                                      dtype=torch.float32).to(DTYPES[case["dtype"]]))
    rng = np.random.Generator(np.random.PCG64(seed))
    parents = np.minimum((rng.random((B, K)) ** 2 * K).astype(np.int32), K - 1)
    if case["inplace"]:
        # caches kept in place: a survivor stays in its slot, the freed slots
        # take copies
        kept = np.zeros((B, K), bool)
        np.put_along_axis(kept, parents, True, 1)
        parents = np.where(kept, np.arange(K, dtype=np.int32), parents)
    return {"caches": caches, "parents": parents}


def _trace_inputs(case, seed):
    T, B, K = case["T"], case["B"], case["K"]
    g = _generator(seed)
    u = torch.rand((T, B, K), generator=g, device="cuda")
    return {"parents": (u * u * K).to(torch.int32).clamp_(max=K - 1),
            "tokens": torch.randint(0, 151936, (T, B, K), generator=g, device="cuda",
                                    dtype=torch.int32)}


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "trace":
        st.update(_trace_inputs(case, seed))
        return st
    if case["op"] == "reorder":
        st.update(_reorder_inputs(case, seed))
        st["parents"] = torch.from_numpy(st["parents"]).cuda()
        st["views"] = [c[:, :, :, :case["length"]] for c in st["caches"]]
        if not case["inplace"]:
            st["out"] = [torch.zeros_like(c)[:, :, :, :case["length"]] for c in st["caches"]]
        return st
    inp = _select_inputs(case, seed)
    st["logits"], st["scores"] = inp["logits"], inp["scores"]
    edges, S, V = inp["edges"], case["S"], case["V"]
    if own:
        fa, table = _table(case, edges, inp["accept"])
        st["table"] = table
        st["beams"] = fa.BeamBuffers(table, case["B"], case["K"])
        st["beams"].scores.copy_(inp["scores"])
        st["beams"].states.copy_(_words(torch.from_numpy(inp["sets"]).cuda()))
        st["out"] = fa.BeamBuffers(table, case["B"], case["K"])
        st["lookahead"] = fa.beam_lookahead(table, case["steps"]) if case["steps"] else None
        return st
    r = (_reach(edges, inp["accept"], S, case["steps"] - 1) if case["steps"]
         else np.ones(S, bool))
    st["reach"] = torch.from_numpy(r).cuda()
    if case["kind"] == "nfa":
        # every (source, token, target) of the automaton
        n = [e[2].size for e in edges]
        st["src"] = torch.from_numpy(np.repeat([e[0] for e in edges], n)).cuda()
        st["dst"] = torch.from_numpy(np.repeat([e[1] for e in edges], n)).cuda()
        st["tok"] = torch.from_numpy(np.concatenate([e[2] for e in edges])).cuda()
        st["sets"] = torch.from_numpy(inp["sets"]).cuda()
    else:
        # the transition function, -1 where a token has no edge
        delta = np.full((S, V), -1, np.int16)
        for a, b, lab in edges:
            if case["kind"] == "range":
                delta[a, lab[0]:lab[1]] = b
            else:
                delta[a, lab] = b
        st["delta"] = torch.from_numpy(delta).cuda()
        st["ids"] = torch.from_numpy(inp["ids"]).cuda()
    return st


# -------------------------------------------------------------------- run
def _top(score, K):
    """The K largest of every row, ties to the lower index; their values in
    descending order and their indices."""
    N = score.shape[1]
    kth = torch.topk(score, K).values[:, -1:]
    above, equal = score > kth, score == kth
    left = K - above.sum(-1, keepdim=True)
    take = above | (equal & (torch.cumsum(equal, -1, dtype=torch.int32) <= left))
    rank = torch.where(take, N - torch.arange(N, device=score.device, dtype=torch.int32), 0)
    idx = N - torch.topk(rank, K).values.long()  # ascending
    val, order = torch.sort(score.gather(1, idx), dim=1, descending=True, stable=True)
    return val, idx.gather(1, order)


def _plain_select(st):
    c = st["case"]
    B, K, V, S = c["B"], c["K"], c["V"], c["S"]
    dev = st["logits"].device
    # scores in 64 bits: two beams' candidates may lie closer than 32 resolve
    x = st["logits"].double()
    if c["mode"] == "probs":
        logp = torch.log(x)
    else:
        m = x.amax(-1, keepdim=True)
        logp = x - (torch.log(torch.exp(x - m).sum(-1, keepdim=True)) + m)
    if c["kind"] == "nfa":
        sets = st["sets"].view(B * K, S)
        live = sets[:, st["src"]] & st["reach"][st["dst"]]
        allowed = torch.zeros((B * K, V + 1), dtype=torch.bool, device=dev)
        allowed.scatter_(1, torch.where(live, st["tok"], V), True)
        allowed = allowed[:, :V].reshape(B, K, V)
    else:
        to = st["delta"][st["ids"]]
        allowed = (to >= 0) & st["reach"][to.clamp(min=0).long()]
    score = torch.where(allowed, st["scores"].double()[..., None] + logp, -math.inf)
    val, idx = _top(score.view(B, K * V), K)
    found = val > -math.inf
    slots = torch.arange(K, device=dev)
    parents = torch.where(found, idx // V, slots)
    tokens = torch.where(found, idx % V, -1)
    new = torch.zeros((B, K, S + 1), dtype=torch.bool, device=dev)
    if c["kind"] == "nfa":
        at = live.view(B, K, -1).gather(1, parents[..., None].expand(-1, -1, live.shape[1]))
        at = at & (st["tok"] == tokens[..., None])
        new.scatter_(2, torch.where(at, st["dst"], S), True)
    else:
        s = st["delta"][st["ids"].gather(1, parents), tokens.clamp(min=0)].long()
        new.scatter_(2, torch.where(found, s, S)[..., None], True)
    return {"scores": val.float(), "tokens": tokens.int(), "parents": parents.int(),
            "states": _words(new[..., :S])}


def _plain_reorder(st):
    rows = torch.arange(st["parents"].shape[0], device="cuda")[:, None]
    par = st["parents"].long()
    for v, o in zip(st["views"], st.get("out", st["views"])):
        o.copy_(v[rows, par])
    return st["out"] if "out" in st else st["caches"]


def _plain_trace(st):
    T, B, K = st["tokens"].shape
    out = torch.empty((B, K, T), dtype=torch.int32, device="cuda")
    j = torch.arange(K, device="cuda").expand(B, K)
    for t in range(T - 1, -1, -1):
        out[:, :, t] = st["tokens"][t].gather(1, j)
        j = st["parents"][t].long().gather(1, j)
    return out


def run(st):
    c = st["case"]
    if own:
        import constrained_decoding_diffusion_amd as fa
        if c["op"] == "trace":
            return fa.beam_trace(st["tokens"], st["parents"])
        if c["op"] == "reorder":
            fa.beam_reorder(st["views"], st["parents"], out=st.get("out"))
            return st["out"] if "out" in st else st["caches"]
        mode = fa.FA_BEAM_PROBS if c["mode"] == "probs" else fa.FA_BEAM_LOGITS
        out = fa.beam_select(st["table"], st["logits"], st["beams"], out=st["out"], mode=mode,
                             steps_left=c["steps"], lookahead=st["lookahead"])
        return {"scores": out.scores, "tokens": out.tokens, "parents": out.parents,
                "states": out.states}
    if c["op"] == "trace":
        return _plain_trace(st)
    if c["op"] == "reorder":
        return _plain_reorder(st)
    return _plain_select(st)


# ------------------------------------------------------------------- work
def work(case):
    if case["op"] == "trace":
        return {"bytes": 12 * case["T"] * case["B"] * case["K"], "flops": 0}
    if case["op"] == "reorder":
        B, K = case["B"], case["K"]
        item = case["tensors"] * case["heads"] * case["length"] * case["dim"] * SIZE[case["dtype"]]
        # parents drawn as floor(K u^2): the expected number of distinct ones
        kept = sum(1 - (1 - (math.sqrt((j + 1) / K) - math.sqrt(j / K))) ** K for j in range(K))
        # in place the freed slots alone are written, out of place all are
        moved = (K - kept) if case["inplace"] else K
        read = min(kept, moved) if case["inplace"] else kept
        return {"bytes": int(B * item * (moved + read)), "flops": 0}
    B, K, V, W = case["B"], case["K"], case["V"], (case["S"] + 31) // 32
    rows = B if case["mode"] == "probs" or case["fresh"] else B * K
    live = B if case["fresh"] else B * K
    return {"bytes": rows * V * SIZE[case["dtype"]] + live * 4 * W + B * K * (4 * W + 16),
            "flops": 3 * live * V}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    if case["op"] != "select":
        return None
    B, K, V, S = case["B"], case["K"], case["V"], case["S"]
    inp = _select_inputs(case, seed)
    reach = _reach(inp["edges"], inp["accept"], S, case["steps"] - 1) if case["steps"] else None
    out_of = {}
    for a, b, lab in inp["edges"]:
        if reach is None or reach[b]:
            out_of.setdefault(a, []).append((b, lab))
    scores = np.full((B, K), -np.inf)
    tokens = np.full((B, K), -1, np.int32)
    parents = np.tile(np.arange(K, dtype=np.int32), (B, 1))
    W = (S + 31) // 32
    states = np.zeros((B, K, W), np.int64)
    start = inp["scores"].double().cpu().numpy()
    for b in range(B):
        x = inp["logits"][b].float().cpu().numpy().astype(np.float64)
        key, place = [], []
        for k in range(K):
            if start[b, k] == -np.inf:
                continue
            may = np.zeros(V, bool)
            for q in np.flatnonzero(inp["sets"][b, k]):
                for _, lab in out_of.get(q, []):
                    may[slice(*lab) if isinstance(lab, tuple) else lab] = True
            v = np.flatnonzero(may)
            with np.errstate(divide="ignore"):
                if case["mode"] == "probs":
                    s = start[b, k] + np.log(x[k, v])
                else:
                    top = x[k].max()
                    s = start[b, k] + (x[k, v] - (np.log(np.exp(x[k] - top).sum()) + top))
            if K < v.size:  # a beam gives K candidates at most (and those that tie with its last)
                near = s >= np.partition(s, v.size - K)[v.size - K]
                s, v = s[near], v[near]
            key.append(s)
            place.append(k * V + v)
        key, place = np.concatenate(key), np.concatenate(place)
        order = np.lexsort((place, -key))[:K]
        order = order[key[order] > -np.inf]
        for j, o in enumerate(order):
            scores[b, j] = key[o]
            parents[b, j], tokens[b, j] = divmod(int(place[o]), V)
            for q in np.flatnonzero(inp["sets"][b, parents[b, j]]):
                for to, lab in out_of.get(q, []):
                    t = tokens[b, j]
                    if lab[0] <= t < lab[1] if isinstance(lab, tuple) else t in lab:
                        states[b, j, to // 32] |= 1 << (to % 32)
    return {"scores": scores, "tokens": tokens, "parents": parents,
            "states": states.astype(np.uint32).view(np.int32)}
