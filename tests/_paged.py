"""A paged cache built token by token, and its operators restated in 64 bits over
plain lists of tokens; used by the tests of the paged K/V cache.

Tolerances, derived from the arithmetic of the kernels (u = 2^-23, one unit in
the last place of an f32 sum, which the tensor cores may truncate):
  * a logit is a sum of 128 products: its error is at most
    e = 144 u |scale| sum_d |q_d k_jd|, the largest over the visible tokens
    (16 more for the scaling and the splits of its operands);
  * a weight exp(l - max) has a relative error of at most 2 e + 16 u (its own
    logit, the maximum's, the exponential and its argument's rounding);
  * numerator and denominator are f32 sums of up to n terms, n u each;
so an f32 output is off by at most (4 e + (2 n + 64) u) * sum_j w_j |v_j|, a
log-sum-exp by 2 e + (n + 64) u + 2 u |lse|, a weight by (4 e + (n + 64) u) w.
The prompt form rounds the weights and the output to bf16 besides: 2^-8 of
sum_j w_j |v_j| and 2^-8 of the output.
"""
import numpy as np
import torch

U = 2.0 ** -23
D = 128


def make(lens, G, page, seed=0, layout="head", spare=3, slack=1, poison=True, device="cuda", cap_pages=None):
    """A cache of R = len(lens) requests with lens[r] random tokens in pages in no order. Rows that hold no
    token are NaN, table entries behind the last page are garbage. -> (k, v, table, n), k and v as
    [P][G][page][D] views of the layout."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    need = [-(-x // page) for x in lens]
    mp = cap_pages or max(need) + slack
    total = sum(need) + spare
    fill = float("nan") if poison else 0.0
    shape = (total, G, page, D) if layout == "head" else (total, page, G, D)
    if layout == "both":  # K and V of a page side by side in one array
        both = torch.full((total, 2, page, G, D), fill, dtype=torch.bfloat16)
        k, v = (both[:, i].transpose(1, 2) for i in (0, 1))
    else:
        k, v = (torch.full(shape, fill, dtype=torch.bfloat16) for _ in range(2))
        if layout == "token":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(total, generator=g)
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (R, mp), generator=g).to(torch.int32)
    ks = torch.exp(0.7 * torch.randn(G, 1, D, generator=g))
    at = 0
    for r, x in enumerate(lens):
        for p in range(need[r]):
            table[r, p] = int(order[at])
            m = min(page, x - p * page)
            k[order[at], :, :m] = (torch.randn(G, m, D, generator=g) * ks).to(torch.bfloat16)
            v[order[at], :, :m] = torch.randn(G, m, D, generator=g).to(torch.bfloat16)
            at += 1
    n = torch.tensor(lens, dtype=torch.int32)
    if layout == "both":
        dev = both.to(device)
        k, v = (dev[:, i].transpose(1, 2) for i in (0, 1))
    elif layout == "token":
        k, v = (t.transpose(1, 2).to(device).transpose(1, 2) for t in (k, v))
    else:
        k, v = k.to(device), v.to(device)
    return k, v, table.to(device), n.to(device)


def tokens(pool, table, r, n):
    """Request r's first n rows in order, f64 [n][G][D]."""
    page = pool.shape[2]
    out = [pool[int(table[r, p])].permute(1, 0, 2).double() for p in range(-(-n // page))]
    return torch.cat(out)[:n] if out else torch.zeros(0, pool.shape[1], D, dtype=torch.float64, device=pool.device)


def visible(p, window, sinks):
    """The tokens that the one at position p sees."""
    j = np.arange(max(p + 1, 0))
    return j if not window else j[(j < sinks) | (j > p - window)]


def attend(q, K, V, scale):
    """q f64 [..., D], K, V f64 [n][D] -> out, lse, weights [..., n], and the error bound e of a logit."""
    if K.shape[0] == 0:
        z = torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
        return torch.zeros_like(q), z - float("inf"), torch.zeros(*q.shape[:-1], 0, dtype=torch.float64,
                                                                   device=q.device), z, torch.zeros_like(q)
    l = q @ K.T * scale
    lse = torch.logsumexp(l, -1)
    w = torch.exp(l - lse.unsqueeze(-1))
    e = 144 * U * abs(scale) * (q.abs() @ K.abs().T).amax(-1)
    return w @ V, lse, w, e, w @ V.abs()


def check_decode(out, lse, q, k, v, table, lens, window, sinks, scale, mass=None, mass_out=None):
    """One decode call against the definition; mass is what it was before, mass_out after."""
    R, G, H, _ = q.shape
    for r in range(R):
        vis = torch.from_numpy(visible(lens[r] - 1, window, sinks)).to(q.device)
        K, V = tokens(k, table, r, lens[r])[vis], tokens(v, table, r, lens[r])[vis]
        n = len(vis)
        for g in range(G):
            o, ls, w, e, va = attend(q[r, g].double(), K[:, g], V[:, g], scale)
            if n == 0:
                assert torch.equal(out[r, g], torch.zeros_like(out[r, g])), (r, g)
                assert bool(torch.isneginf(lse[r, g]).all()), (r, g)
            else:
                tol = (4 * e.unsqueeze(-1) + (2 * n + 64) * U) * va
                err = (out[r, g].double() - o).abs()
                assert bool((err <= tol).all()), (r, g, float((err / tol).max()))
                # and as a whole far inside the worst case
                assert float(err.norm() / o.norm()) < 2e-5, (r, g, float(err.norm() / o.norm()))
                ltol = 2 * e + (n + 64) * U + 2 * U * ls.abs()
                assert bool(((lse[r, g].double() - ls).abs() <= ltol).all()), (r, g)
            if mass is not None:
                want = mass[r, g].double().clone()
                want[vis] += w.sum(0)
                tol = torch.full_like(want, 0.0)
                tol[vis] = ((4 * e.unsqueeze(-1) + (n + 64) * U) * w).sum(0) + 2 * U * want[vis].abs()
                err = (mass_out[r, g].double() - want).abs()
                err[torch.isnan(want) & torch.isnan(mass_out[r, g].double())] = 0  # untouched entries
                assert bool((err <= tol).all()), (r, g, int((err > tol).sum()))


def check_prompt(out, lse, q, cu, k, v, table, lens, window, sinks, scale, G):
    """One prompt call against the definition, query by query."""
    H = q.shape[1] // G
    for r in range(len(lens)):
        a, b = cu[r], cu[r + 1]
        K, V = tokens(k, table, r, lens[r]), tokens(v, table, r, lens[r])
        for g in range(G):
            qg = q[a:b, g * H:(g + 1) * H].double()  # [c][H][D]
            p = torch.arange(lens[r] - (b - a), lens[r], device=q.device).view(-1, 1, 1)
            j = torch.arange(lens[r], device=q.device)
            ok = j <= p
            if window:
                ok = ok & ((j < sinks) | (j > p - window))
            l = (qg @ K[:, g].T * scale).masked_fill(~ok, float("-inf"))
            e = 144 * U * abs(scale) * (qg.abs() @ K[:, g].abs().T).masked_fill(~ok, 0.0).amax(-1) \
                if lens[r] else torch.zeros(b - a, H, dtype=torch.float64, device=q.device)
            ls = torch.logsumexp(l, -1)
            w = torch.where(ok, torch.exp(l - ls.unsqueeze(-1)), 0.0)
            o, va = w @ V[:, g], w @ V[:, g].abs()
            n = ok.sum(-1).double()
            got, gl = out[a:b, g * H:(g + 1) * H].double(), lse[a:b, g * H:(g + 1) * H].double()
            none = n.expand_as(ls) == 0
            assert bool((got[none] == 0).all()) and bool(torch.isneginf(gl[none]).all())
            f32 = (4 * e + (2 * n + 64) * U).unsqueeze(-1) * va
            tol = 2.0 ** -8 * (va + o.abs()) * (1 + 2.0 ** -7) + f32
            err = (got - o).abs()
            assert bool((err <= tol).all()), (r, g, float((err / tol).nan_to_num(0).max()))
            ltol = 2 * e + (n + 64) * U + 2 * U * ls.abs()
            assert bool(((gl - ls).abs()[~none] <= ltol.expand_as(ls)[~none]).all()), (r, g)


def evict(mass, pos, n, seen, budget, sinks, recent):
    """The slots that the first min(n, budget) slots' tokens come from, by the definition; numpy, one row."""
    if n <= budget:
        return np.arange(n)
    slots = np.arange(n)
    sure = (pos[:n] < sinks) | (pos[:n] >= seen - recent)
    m = np.where(np.isnan(mass[:n]), -np.inf, mass[:n].astype(np.float64))
    m[sure] = 0  # alike: only their slots order them
    nan = np.isnan(mass[:n]) & ~sure
    rank = np.lexsort((slots, nan, -m, ~sure))
    kept = np.zeros(n, bool)
    kept[rank[:budget]] = True
    src = np.arange(budget)
    src[~kept[:budget]] = slots[budget:][kept[budget:]]
    return src
