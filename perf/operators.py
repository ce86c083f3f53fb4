"""Measured cases of the sampling and page-pool operators.

``sample_tokens`` draws a token per row of logits under a temperature, top-k,
top-p and min-p from given uniforms and can hand out the distribution it drew
from.  ``kv_pages_copy``, ``kv_pages_fork``, ``kv_pages_resize`` and
``kv_pages_compact`` manage the pages of the paged latent cache: copying
pages, forking a request into continuations that share its pages, giving
requests the pages of their new lengths (or taking them back) and closing the
holes of a fragmented pool.

With ``own`` false a pass computes an operator in plain torch operations, with
``own`` true through the package's entry points.  Pool contents are changed in
place; the tables, counts and lengths go into new tensors, so a pass can be
repeated on the same state.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
PAGE = 64     # rows of a page
WIDTH = 512   # latent width
TYPES = {"bf16": torch.bfloat16, "fp8": torch.uint8, "fp32": torch.float32}
#: a token below this fraction of the row's largest weight is outside the support
SUPPORT = 2.0 ** -40


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one request decoding alone with the usual chat settings: latency
        dict(name="sample-one", op="sample", T=1, V=163840, pad=0, dtype="fp32", probs=False, mode="k50p90"),
        # the drafts of 32 requests, with the distribution that sampled verification tests them against
        dict(name="sample-draft-probs", op="sample", T=32, V=163840, pad=0, dtype="fp32", probs=True, mode="p95"),
        # a mixed batch, each row with its request's own settings (greedy rows among them), a vocabulary
        # of odd size in padded bf16 rows
        dict(name="sample-mixed-odd", op="sample", T=67, V=32003, pad=61, dtype="bf16", probs=False, mode="mixed"),
        # a full decode batch over the whole vocabulary with a min-p floor
        dict(name="sample-batch", op="sample", T=512, V=163840, pad=0, dtype="fp32", probs=False, mode="minp"),
        # a few pages of one layer (a beam's tails): latency
        dict(name="copy-few", op="copy", L=1, P=256, n=8, dtype="bf16", same=True),
        # requests moved from one pool to another, all layers
        dict(name="copy-layers", op="copy", L=24, P=320, n=256, dtype="bf16", same=False),
        # one prompt forked into three continuations, one layer
        dict(name="fork-one", op="fork", L=1, P=256, R=8, max_pages=24, lo=1024, hi=1536, parents=1, each=3, dtype="bf16"),
        # parallel sampling: 16 prompts, four continuations each, all layers
        dict(name="fork-batch", op="fork", L=24, P=512, R=96, max_pages=24, lo=1024, hi=1536, parents=16, each=4, dtype="bf16"),
        # the verify step's page bookkeeping of eight requests: groups appended, rejected tails dropped
        dict(name="resize-step", op="resize", P=256, R=8, max_pages=24, lo=1024, hi=1400),
        # 256 long contexts in a large pool: some finish, some are admitted, the rest grow or shrink
        dict(name="resize-long", op="resize", P=65536, R=256, max_pages=512, lo=8192, hi=30000),
        # a small pool with a third of its pages in use, scattered
        dict(name="compact-small", op="compact", L=1, P=256, R=6, max_pages=24, lo=1024, hi=1536, dtype="bf16"),
        # a pool of eight layers, half of it free in scattered holes
        dict(name="compact-layers", op="compact", L=8, P=1024, R=24, max_pages=24, lo=1024, hi=1536, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "copy", "fork", "resize", "compact"])
    if op == "sample":
        V = _log(rng, 1000, 163840)
        T = _log(rng, 1, 512)
        probs = rng.random() < 0.3
        while T * V * (2 if probs else 1) > 512 * 163840 // 2:
            T = max(1, T // 2)
        return dict(op=op, T=T, V=V, pad=rng.choice([0, 0, rng.randint(1, 200)]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    probs=probs, mode=rng.choice(["k50p90", "p95", "mixed", "minp", "plain", "k1000"]))
    dtype = rng.choice(["bf16", "bf16", "fp8"])
    L = _log(rng, 1, 24)
    if op == "copy":
        n = _log(rng, 1, 256)
        return dict(op=op, L=L, P=2 * n + rng.randint(1, 99), n=n, dtype=dtype, same=rng.random() < 0.5)
    if op == "fork":
        parents, each = _log(rng, 1, 16), rng.randint(1, 4)
        max_pages = rng.randint(2, 24)
        hi = max_pages * PAGE
        R = parents * (1 + each) + rng.randint(0, 9)
        return dict(op=op, L=L, P=max(64, parents * max_pages + parents * each + rng.randint(0, 40)), R=R, max_pages=max_pages,
                    lo=rng.randint(1, hi), hi=hi, parents=parents, each=each, dtype=dtype)
    if op == "resize":
        R, max_pages = _log(rng, 1, 256), _log(rng, 2, 512)
        cap = max_pages * PAGE
        return dict(op=op, P=max(64, min(65536, R * max_pages // rng.choice([1, 2]) + rng.randint(0, 99))), R=R, max_pages=max_pages,
                    lo=max(1, cap // 8), hi=max(1, cap * 3 // 4))
    P = _log(rng, 64, 1024)
    max_pages = rng.randint(2, 24)
    R = max(1, P // (2 * max_pages))
    return dict(op=op, L=min(L, 8), P=P, R=R, max_pages=max_pages, lo=max(1, max_pages * PAGE // 2), hi=max_pages * PAGE, dtype=dtype)


# ---------------------------------------------------------------- inputs
def _settings(case, g):
    """Per-row temperature, top_k, top_p, min_p: a number for the whole batch or a tensor of one value per row."""
    T, mode = case["T"], case["mode"]
    if mode == "k50p90":
        return 0.8, 50, 0.9, 0.0
    if mode == "p95":
        return 1.0, 0, 0.95, 0.0
    if mode == "minp":
        return 0.9, 0, 1.0, 0.05
    if mode == "plain":
        return 1.0, 0, 1.0, 0.0
    if mode == "k1000":
        return 1.1, 1000, 1.0, 0.0
    r = torch.rand((4, T), generator=g, device=DEV)
    temperature = torch.where(r[0] < 0.15, torch.zeros_like(r[0]), 0.5 + r[0])
    top_k = torch.where(r[1] < 0.4, torch.zeros_like(r[1]), 1 + r[1] * 100).to(torch.int32)
    top_p = torch.where(r[2] < 0.4, torch.ones_like(r[2]), 0.4 + 0.59 * r[2])
    min_p = torch.where(r[3] < 0.5, torch.zeros_like(r[3]), 0.1 * r[3])
    return temperature, top_k, top_p, min_p


def _prepare_sample(case, g):
    T, V = case["T"], case["V"]
    wide = torch.empty((T, V + case["pad"]), dtype=torch.float32, device=DEV)
    wide.normal_(generator=g)
    # rows from flat to peaked: a bulk of spread 1..3 and some tokens that stand out of it
    spread = 1.0 + 2.0 * torch.rand((T, 1), generator=g, device=DEV)
    wide *= spread
    n = min(V, 24)
    at = torch.randint(0, V, (T, n), generator=g, device=DEV)
    high = 3.0 * spread + 12.0 * torch.rand((T, n), generator=g, device=DEV)
    wide.scatter_(1, at, high)
    wide = wide.to(TYPES[case["dtype"]])
    return dict(case=case, logits=wide[:, :V], uniforms=torch.rand(T, generator=g, device=DEV), settings=_settings(case, g))


def _pool(case, g, pages):
    shape = (case["L"], pages, PAGE, WIDTH)
    if case["dtype"] == "fp8":
        return torch.randint(0, 120, shape, generator=g, device=DEV, dtype=torch.uint8)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _lengths(case, g, n):
    return torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g, device=DEV)


def _tables(case, g, lens, shared):
    """Tables of requests that hold scattered pages: (ref_counts, block_table).  With `shared`, every odd request
    shares the full pages of the first half of the shorter length with the request before it."""
    P, R, mp = case["P"], case["R"], case["max_pages"]
    held = (lens + PAGE - 1) // PAGE
    held = torch.where(held.cumsum(0) <= P, held, torch.zeros_like(held))  # as many as the pool holds
    j = torch.arange(mp, device=DEV)
    mine = j[None, :] < held[:, None]
    order = torch.randperm(P, generator=g, device=DEV)
    first = held.cumsum(0) - held
    table = torch.where(mine, order[(first[:, None] + j[None, :]).clamp(max=P - 1)], torch.full_like(j, -1)[None, :])
    if shared and R > 1:
        prev = torch.roll(table, 1, 0)
        both = torch.minimum(lens, torch.roll(lens, 1)) // PAGE // 2
        odd = (torch.arange(R, device=DEV) % 2 == 1) & (held > 0) & (torch.roll(held, 1) > 0)
        take = odd[:, None] & (j[None, :] < both[:, None])
        table = torch.where(take, prev, table)
    counts = torch.zeros(P + 1, dtype=torch.int64, device=DEV)
    counts.scatter_add_(0, torch.where(table >= 0, table, torch.full_like(table, P)).reshape(-1), torch.ones(R * mp, dtype=torch.int64, device=DEV))
    lens = torch.where(held > 0, lens, torch.zeros_like(lens))
    return counts[:P].to(torch.int32), table.to(torch.int32), lens.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 17)
    op = case["op"]
    if op == "sample":
        return _prepare_sample(case, g)
    if op == "copy":
        n, P = case["n"], case["P"]
        src = _pool(case, g, P)
        if case["same"]:
            ids = torch.randperm(P, generator=g, device=DEV)[:2 * n].to(torch.int32)
            return dict(case=case, src=src, dst=src, src_ids=ids[:n].contiguous(), dst_ids=ids[n:].contiguous())
        dst = _pool(case, g, P)
        return dict(case=case, src=src, dst=dst, src_ids=torch.randperm(P, generator=g, device=DEV)[:n].to(torch.int32),
                    dst_ids=torch.randperm(P, generator=g, device=DEV)[:n].to(torch.int32))
    R = case["R"]
    if op == "fork":
        n = case["parents"]
        lens = torch.zeros(R, dtype=torch.int64, device=DEV)
        lens[:n] = _lengths(case, g, n)
        refs, table, lens = _tables(case, g, lens, False)
        parents = torch.arange(n, device=DEV).repeat_interleave(case["each"]).to(torch.int32)
        children = (n + torch.randperm(R - n, generator=g, device=DEV)[:n * case["each"]]).to(torch.int32)
        return dict(case=case, pool=_pool(case, g, case["P"]), refs=refs, table=table, lens=lens, parents=parents, children=children)
    lens = _lengths(case, g, R)
    if op == "resize":
        cap = case["max_pages"] * PAGE
        lens = torch.where(torch.rand(R, generator=g, device=DEV) < 0.1, torch.zeros_like(lens), lens)  # empty slots
        refs, table, lens = _tables(case, g, lens, True)
        kind = torch.rand(R, generator=g, device=DEV)
        step = torch.randint(1, 9, (R,), generator=g, device=DEV)
        new = lens.long() + step                                                                # a verify group appended
        new = torch.where(kind < 0.4, (lens - step).clamp(min=0).long(), new)                   # a rejected tail dropped
        new = torch.where(kind < 0.1, torch.zeros_like(new), new)                               # finished
        new = torch.where(lens == 0, torch.randint(0, cap // 2 + 1, (R,), generator=g, device=DEV), new)  # admitted
        return dict(case=case, refs=refs, table=table, lens=lens, new=new.clamp(max=cap).to(torch.int32))
    refs, table, lens = _tables(case, g, lens, True)
    return dict(case=case, pool=_pool(case, g, case["P"]), refs=refs, table=table, lens=lens)


# ---------------------------------------------------------------- the plain forms
def _rows(v, T, dtype):
    return v.to(dtype) if isinstance(v, torch.Tensor) else torch.full((T,), v, dtype=dtype, device=DEV)


def _plain_sample(s):
    x = s["logits"].float()
    T, V = x.shape
    temperature, top_k, top_p, min_p = s["settings"]
    # the settings as the entry point takes them: fp32 numbers
    tau = _rows(temperature, T, torch.float32).double()[:, None]
    p = _rows(top_p, T, torch.float32).double()[:, None]
    floor = _rows(min_p, T, torch.float32).double()[:, None]
    k = _rows(top_k, T, torch.int64)
    k = torch.where((k <= 0) | (k > V), torch.full_like(k, V), k)[:, None]
    greedy = tau <= 0
    tau = torch.where(greedy, torch.ones_like(tau), tau)
    m = x.amax(1, keepdim=True)
    w = ((x.double() - m.double()) / tau).exp()
    xs = x.sort(dim=1, descending=True)[0]
    border_k = xs.gather(1, k - 1)
    ws = torch.where(xs >= border_k, ((xs.double() - m.double()) / tau).exp(), torch.zeros_like(w))
    cum = ws.cumsum(1)
    at = (cum < p * cum[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
    border_p = torch.where(p >= 1, torch.full_like(m, -math.inf), xs.gather(1, at))
    keep = (x >= border_k) & (x >= border_p) & (w >= floor) & (w >= SUPPORT)
    w = torch.where(keep, w, torch.zeros_like(w))
    cum = w.cumsum(1)
    total = cum[:, -1:]
    drawn = (cum <= s["uniforms"].double()[:, None] * total).sum(1).clamp(max=V - 1)
    ids = torch.arange(V, device=x.device)[None, :]
    best = torch.where(x == m, ids, torch.full_like(ids, V)).amin(1)
    tokens = torch.where(greedy[:, 0], best, drawn).to(torch.int32)
    if not s["case"]["probs"]:
        return tokens
    probs = torch.where(greedy, (ids == best[:, None]).double(), w / total)
    return tokens, probs.float()


def _plain_copy(s):
    s["dst"][:, s["dst_ids"].long()] = s["src"][:, s["src_ids"].long()]
    return s["dst"]


def _free_list(refs):
    """The free pages in ascending order, then zeros, and their number."""
    P = refs.shape[0]
    free = refs == 0
    rank = free.long().cumsum(0) - 1
    ids = torch.arange(P, device=refs.device)
    return torch.zeros(P + 1, dtype=torch.int64, device=refs.device).scatter_(0, torch.where(free, rank, torch.full_like(rank, P)), ids), free.sum()


def _bump(refs, ids, mask, by):
    """refs with `by` added at ids[mask]."""
    P = refs.shape[0]
    at = torch.where(mask, ids.long(), torch.full_like(ids.long(), P)).reshape(-1)
    wide = torch.cat([refs.long(), refs.new_zeros(1).long()])
    return wide.scatter_add_(0, at, torch.full_like(at, by))[:P].to(torch.int32)


def _plain_fork(s):
    refs, table, lens, pool = s["refs"], s["table"], s["lens"], s["pool"]
    mp = table.shape[1]
    parents, children = s["parents"].long(), s["children"].long()
    plen = lens[parents].long()
    full, tail = plen // PAGE, plen % PAGE
    has = tail > 0
    j = torch.arange(mp, device=table.device)[None, :]
    prow = table[parents]
    shared = j < full[:, None]
    pages, free = _free_list(refs)
    rank = has.long().cumsum(0) - has.long()
    done = ~has | (rank < free)
    new = pages[rank]
    take = has & done
    old = prow.gather(1, full.clamp(max=mp - 1)[:, None])[:, 0].long()
    crow = torch.where(shared & done[:, None], prow, table[children])
    crow = torch.where((j == full[:, None]) & take[:, None], new[:, None].to(torch.int32), crow)
    table2, lens2 = table.clone(), lens.clone()
    table2[children] = crow
    lens2[children] = torch.where(done, plen.to(torch.int32), lens[children])
    refs2 = _bump(_bump(refs, prow, shared & done[:, None], 1), new, take, 1)
    # the rows in use of each tail page
    rows = torch.arange(PAGE, device=table.device)[None, :] < tail[:, None]
    to = torch.where(take, new, prow[:, 0].long())  # a fork without a tail copies a page of its parent onto itself
    here = torch.where(take[:, None] & rows, old[:, None], to[:, None])
    r = torch.arange(PAGE, device=table.device)[None, :].expand_as(rows)
    pool[:, to[:, None], r] = pool[:, here, r]
    return pool, refs2, table2, lens2


def _plain_resize(s):
    refs, table, lens, new = s["refs"], s["table"], s["lens"].long(), s["new"].long()
    mp = table.shape[1]
    have, want = (lens + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    j = torch.arange(mp, device=table.device)[None, :]
    drop = (j >= want[:, None]) & (j < have[:, None])
    refs2 = _bump(refs, table, drop, -1)
    table2 = torch.where(drop, torch.full_like(table, -1), table)
    need = (want - have).clamp(min=0)
    before = need.cumsum(0) - need
    pages, free = _free_list(refs2)
    fits = (need == 0) | (before + need <= free)
    grow = (j >= have[:, None]) & (j < want[:, None]) & fits[:, None]
    page = pages[(before[:, None] + j - have[:, None]).clamp(min=0, max=pages.shape[0] - 1)]
    table2 = torch.where(grow, page.to(torch.int32), table2)
    refs2 = _bump(refs2, page, grow, 1)
    return refs2, table2, torch.where(fits, new, lens).to(torch.int32)


def _plain_compact(s):
    refs, table, lens, pool = s["refs"], s["table"], s["lens"].long(), s["pool"]
    P, mp = refs.shape[0], table.shape[1]
    live = refs != 0
    n = live.sum()
    ids = torch.arange(P, device=refs.device)
    hole, high = ~live & (ids < n), live & (ids >= n)
    holes = torch.full((P + 1,), -1, dtype=torch.int64, device=refs.device)
    holes.scatter_(0, torch.where(hole, hole.long().cumsum(0) - 1, torch.full_like(ids, P)), ids)
    to = torch.where(high, holes[(high.long().cumsum(0) - 1).clamp(min=0)], ids)
    page_map = torch.where(live, to, torch.full_like(ids, -1))
    at = torch.where(live, to, torch.full_like(ids, P))
    refs2 = torch.zeros(P + 1, dtype=torch.int32, device=refs.device).scatter_(0, at, refs)[:P]
    held = torch.arange(mp, device=refs.device)[None, :] < ((lens + PAGE - 1) // PAGE)[:, None]
    table2 = torch.where(held, page_map[table.long().clamp(min=0)].to(torch.int32), table)
    # at most half of the pages move; the rest of the list copies the last page onto itself
    half = P // 2
    src = torch.full((P + 1,), P - 1, dtype=torch.int64, device=refs.device)
    src.scatter_(0, torch.where(high, high.long().cumsum(0) - 1, torch.full_like(ids, P)), ids)
    dst = torch.where(ids < high.sum(), holes[:P], torch.full_like(ids, P - 1))
    src = torch.where(ids < high.sum(), src[:P], torch.full_like(ids, P - 1))
    pool[:, dst[:half]] = pool[:, src[:half]]
    return pool, refs2, table2, page_map.to(torch.int32), n.to(torch.int32).reshape(1)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"sample": _plain_sample, "copy": _plain_copy, "fork": _plain_fork, "resize": _plain_resize, "compact": _plain_compact}[op](state)
    import speculative_decoding_verify_mla_gb300 as sv
    if op == "sample":
        temperature, top_k, top_p, min_p = state["settings"]
        return sv.sample_tokens(state["logits"], state["uniforms"], temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                                return_probs=state["case"]["probs"])
    if op == "copy":
        return sv.kv_pages_copy(state["src"], state["dst"], state["src_ids"], state["dst_ids"])
    if op == "fork":
        refs, table, lens = sv.kv_pages_fork(state["pool"], state["refs"], state["table"], state["lens"], state["parents"], state["children"])
        return state["pool"], refs, table, lens
    if op == "resize":
        return sv.kv_pages_resize(state["refs"], state["table"], state["lens"], state["new"])
    refs, table, page_map, live = sv.kv_pages_compact(state["pool"], state["refs"], state["table"], state["lens"])
    return state["pool"], refs, table, page_map, live


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "sample":
        each = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["T"] * (case["V"] * (each + (4 if case["probs"] else 0)) + 8), "flops": 0}
    if op == "resize":
        # the counts, the tables and the lengths, in and out
        return {"bytes": 8 * (case["P"] + case["R"] * (case["max_pages"] + 1)) + 4 * case["R"], "flops": 0}
    row = WIDTH * (1 if case["dtype"] == "fp8" else 2)
    if op == "copy":
        return {"bytes": 2 * case["L"] * case["n"] * PAGE * row + 8 * case["n"], "flops": 0}
    meta = 8 * (case["P"] + case["R"] * (case["max_pages"] + 1))
    if op == "fork":
        # a tail page is half full on average
        n = case["parents"] * case["each"]
        return {"bytes": 2 * case["L"] * n * (PAGE // 2) * row + meta + 8 * n, "flops": 0}
    # live pages scattered evenly: those above the live count move into the holes below it
    live = min(1.0, case["R"] * ((case["lo"] + case["hi"]) / 2 / PAGE + 0.5) * 0.75 / case["P"])
    return {"bytes": 2 * case["L"] * case["P"] * live * (1 - live) * PAGE * row + meta + 4 * case["P"], "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits, one row or request after the other
def _exact_sample(case, s):
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    T, V = x.shape
    conf = [(v.cpu().numpy() if isinstance(v, torch.Tensor) else np.full(T, v, t)) for v, t in zip(s["settings"], (np.float32, np.int64, np.float32, np.float32))]
    u = s["uniforms"].cpu().numpy().astype(np.float64)
    tokens, probs = np.zeros(T, np.int32), (np.zeros((T, V)) if case["probs"] else None)
    for t in range(T):
        tau, k, p, low = float(conf[0][t]), int(conf[1][t]), float(conf[2][t]), float(conf[3][t])
        row = x[t]
        top = row.max()
        if tau <= 0:
            tokens[t] = int(np.flatnonzero(row == top)[0])
            if probs is not None:
                probs[t, tokens[t]] = 1.0
            continue
        weight = np.exp((row - top) / tau)
        kept = weight >= max(low, SUPPORT)
        if 0 < k < V:
            kept &= row >= np.partition(row, V - k)[V - k]
        if p < 1:
            # over what top-k leaves, whatever min-p says
            pool = np.sort(row[row >= np.partition(row, V - k)[V - k]] if 0 < k < V else row)[::-1]
            mass = np.cumsum(np.exp((pool - top) / tau))
            kept &= row >= pool[min(len(pool) - 1, int(np.searchsorted(mass, p * mass[-1])))]
        ids = np.flatnonzero(kept)
        mass = np.cumsum(weight[ids])
        tokens[t] = ids[min(len(ids) - 1, int(np.searchsorted(mass, u[t] * mass[-1], side="right")))]
        if probs is not None:
            probs[t, ids] = weight[ids] / mass[-1]
    return tokens if probs is None else (tokens, probs)


def _exact_pages(case, s):
    op = case["op"]
    if op == "copy":
        out = s["dst"].cpu().clone()
        src = s["src"].cpu()
        for a, b in zip(s["src_ids"].tolist(), s["dst_ids"].tolist()):
            out[:, b] = src[:, a]
        return out
    refs, lens = s["refs"].cpu().numpy().copy(), s["lens"].cpu().numpy().copy()
    table = s["table"].cpu().numpy().copy()
    if op == "resize":
        new = s["new"].cpu().numpy()
        for r in range(len(lens)):
            for j in range(-(-int(new[r]) // PAGE), -(-int(lens[r]) // PAGE)):
                refs[table[r, j]] -= 1
                table[r, j] = -1
        free = [int(q) for q in np.flatnonzero(refs == 0)]
        asked = 0
        for r in range(len(lens)):
            have, want = -(-int(lens[r]) // PAGE), -(-int(new[r]) // PAGE)
            first, asked = asked, asked + max(0, want - have)
            if want > have and asked > len(free):
                continue
            for j in range(have, want):
                table[r, j] = free[first + j - have]
                refs[table[r, j]] = 1
            lens[r] = new[r]
        return refs, table, lens
    pool = s["pool"].cpu().clone()
    if op == "fork":
        free = [int(q) for q in np.flatnonzero(refs == 0)]
        asked = 0
        for a, b in zip(s["parents"].tolist(), s["children"].tolist()):
            full, tail = divmod(int(lens[a]), PAGE)
            if tail:
                asked += 1
                if asked > len(free):
                    continue
                table[b, full] = free[asked - 1]
                refs[free[asked - 1]] = 1
                pool[:, free[asked - 1], :tail] = pool[:, int(table[a, full]), :tail]
            for j in range(full):
                table[b, j] = table[a, j]
                refs[table[a, j]] += 1
            lens[b] = lens[a]
        return pool, refs, table, lens
    live = [int(q) for q in np.flatnonzero(refs)]
    n = len(live)
    gone = {p: p for p in live if p < n}
    gone.update(zip([p for p in live if p >= n], sorted(set(range(n)) - set(live))))
    page_map, refs2 = np.full(len(refs), -1, np.int32), np.zeros_like(refs)
    for p, q in gone.items():
        page_map[p], refs2[q] = q, refs[p]
        if p != q:
            pool[:, q] = pool[:, p]
    for r in range(len(lens)):
        for j in range(-(-int(lens[r]) // PAGE)):
            table[r, j] = page_map[table[r, j]]
    return pool, refs2, table, page_map, np.array([n], np.int32)


def exact(case, seed):
    if not torch.cuda.is_available():
        return None
    s = prepare(case, seed)
    return _exact_sample(case, s) if case["op"] == "sample" else _exact_pages(case, s)
