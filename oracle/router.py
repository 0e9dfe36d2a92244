"""Router: softmax top-k with routed scaling and an optional shared expert,
written out from its definition.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

FlashInfer PR #4287 runs its expert kernel behind a fixed router (real-model
evaluation: the AlphaMoE router held fixed; its companion router PR is named
among the related PRs) and states the two geometries it routes for in its
retained-measurements notes: routed scaling 1.0 with no shared expert, and
routed scaling 2.5 with one shared expert (E=257, top-9 including the shared
one).  The workload descriptions route with softmax over the experts, top-k,
and weights renormalised over the chosen experts.

Readings taken where the pages are silent:
  * the k chosen experts are the k largest logits, compared exactly as FP32
    values (softmax is increasing, so this is the top-k of the
    probabilities without the ties that rounding exp could create); equal
    logits go to the lower expert index; they are listed in that order
    (largest first);
  * weight of a chosen expert i: exp(l_i) / sum over the chosen exp(l_j),
    times the routed scaling factor (the full softmax denominator cancels in
    the renormalisation), computed here in FP64;
  * a shared expert is expert E_routed, appended to every token as route
    slot top_k with weight 1 (the routed scaling applies to routed experts
    only);
  * logits are finite.
"""

import numpy as np


def router_ref(logits, top_k, n_shared=0, routed_scaling=1.0):
    """logits: float32 [M, E_routed].  Returns (ids int32 [M, top_k + n_shared],
    weights float64 [M, top_k + n_shared])."""
    logits = np.asarray(logits, dtype=np.float32)
    M, E = logits.shape
    assert 1 <= top_k <= E and n_shared in (0, 1)
    # descending by value, ascending index among equal values
    order = np.lexsort((np.broadcast_to(np.arange(E), (M, E)), -logits.astype(np.float64)), axis=1)
    ids = order[:, :top_k].astype(np.int32)
    chosen = np.take_along_axis(logits, ids, axis=1).astype(np.float64)
    e = np.exp(chosen - chosen[:, :1])
    w = e / e.sum(axis=1, keepdims=True) * float(np.float32(routed_scaling))
    if n_shared:
        ids = np.concatenate([ids, np.full((M, 1), E, dtype=np.int32)], axis=1)
        w = np.concatenate([w, np.ones((M, 1))], axis=1)
    return ids, w


def route_scored_ref(logits, top_k, score, bias=None, n_group=1, topk_group=1, group_top=2, renorm=True,
                     routed_scaling=1.0, n_shared=0):
    """Routing by scores, token by token, from its definition in FP64.

    s = sigmoid(l) or softmax(l); c = s + bias decides; the topk_group groups of
    n_group with the largest sums of their group_top largest c are kept (ties:
    the lower group); the top_k largest c (ties: the lower expert) are chosen;
    weights s, divided by their sum (renorm), times routed_scaling.  Logits of
    -infinity or NaN and bias of -infinity or NaN are never chosen, +infinity
    logits count as the largest finite FP32 value, unfilled slots hold id -1,
    weight 0.  logits: [M, E] float32 (or narrower values).  Returns (ids int32,
    weights float64), [M, top_k + n_shared]."""
    l = np.minimum(np.asarray(logits, dtype=np.float64), float(np.finfo(np.float32).max))
    M, E = l.shape
    per = E // n_group
    ids = np.full((M, top_k + n_shared), -1, dtype=np.int32)
    w = np.zeros((M, top_k + n_shared))
    for t in range(M):
        ok = l[t] > -np.inf
        s = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[ok] = 1.0 / (1.0 + np.exp(-l[t][ok]))
        elif ok.any():
            s[ok] = np.exp(l[t][ok] - l[t][ok].max())
            s /= s.sum()
        c = np.where(ok, s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64)), -np.inf)
        c = np.where(np.isnan(c), -np.inf, c)
        if topk_group < n_group:
            gs = np.full(n_group, -np.inf)
            for g in range(n_group):
                best = np.sort(c[g * per:(g + 1) * per])[::-1][:group_top]
                best = best[best > -np.inf]
                if len(best):
                    gs[g] = best.sum()
            kept = np.lexsort((np.arange(n_group), -gs))[:topk_group]
            c = np.where(np.isin(np.arange(E) // per, kept), c, -np.inf)
        order = [e for e in np.lexsort((np.arange(E), -c))[:top_k] if c[e] > -np.inf]
        n = len(order)
        ids[t, :n] = order
        v = s[order]
        if renorm and n:
            # as ratios to the largest, which do not underflow together
            z = l[t][order]
            if score == "sigmoid":
                v = np.exp(-np.logaddexp(0.0, -z) + np.logaddexp(0.0, -z.max()))
            else:
                v = np.exp(z - z.max())
            v = v / v.sum()
        w[t, :n] = v * float(np.float32(routed_scaling))
    if n_shared:
        ids[:, top_k] = E
        w[:, top_k] = 1.0
    return ids, w
