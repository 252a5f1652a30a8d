"""The streaming-attention operators in float64 on the CPU, written from their definitions, with the error bounds
that the GPU results are held to.

A frame at position p of its clip sees j <= p with p - j < window, and j < sinks. Bounds: u is half a step of the
inputs' type relative to the value (finfo.eps / 2) and f = 2^-24 that of float32. A score is a float32 sum of dim
products, off by at most (dim + 2) f of the sum of their magnitudes; an exponential's relative error is its
argument's absolute error plus a few f; weights and score gradients are rounded once to the type of the product they
enter (u); sums over n terms in float32 are off by n f of the sum of magnitudes; results are rounded once (u).
"""

import math

import torch

F32 = 2.0 ** -24


def sees(nq, nk, window, sinks):
    """[nq, nk] bool."""
    p = torch.arange(nq)[:, None] + nk - nq
    j = torch.arange(nk)[None]
    s = j <= p
    if window is not None:
        s &= (p - j < window) | (j < sinks)
    return s


def _softmax(x, mask):
    x = x.masked_fill(~mask, -math.inf)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else torch.full((x.shape[0], 1), -math.inf, dtype=x.dtype)
    safe = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - safe)
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(e))
    return w, (torch.log(total) + safe)[:, 0]


def attention(q, k, v, cu_q, cu_k, window, sinks, scale, dout=None):
    """Returns {"out", "lse", ("dq", "dk", "dv")} as (value, bound) pairs, float64 on the CPU."""
    typ = q.dtype
    u = torch.finfo(typ).eps / 2
    q, k, v = (x.double().cpu() for x in (q, k, v))
    hq, hk, dim = q.shape[1], k.shape[1], q.shape[2]
    group = hq // hk
    res = {"out": [torch.zeros_like(q), torch.zeros_like(q)],
           "lse": [torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64),
                   torch.zeros((hq, q.shape[0]), dtype=torch.float64)]}
    if dout is not None:
        dout = dout.double().cpu()
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            res[n] = [torch.zeros_like(x), torch.zeros_like(x)]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if q1 == q0 or k1 == k0:
            continue
        mask = sees(q1 - q0, k1 - k0, window, sinks)
        for h in range(hq):
            c = h // group
            qi, kj, vj = q[q0:q1, h], k[k0:k1, c], v[k0:k1, c]
            x = qi @ kj.t() * scale
            ex = ((dim + 4) * F32 * scale * (qi.abs() @ kj.abs().t()) + 2 * F32 * x.abs()) * mask
            w, lse = _softmax(x, mask)
            n = mask.sum(1, keepdim=True).double()
            ew = w * (ex + ex.amax(1, keepdim=True) + (n + 8) * F32)      # the weight's own error in float32
            out = w @ vj
            eo = (ew + u * w) @ vj.abs() + (n + 4) * F32 * (w @ vj.abs())
            res["out"][0][q0:q1, h], res["out"][1][q0:q1, h] = out, eo + u * (out.abs() + eo)
            res["lse"][0][h, q0:q1] = lse
            res["lse"][1][h, q0:q1] = ex.amax(1) + ((n + 8) * F32)[:, 0] + 4 * F32 * torch.nan_to_num(lse.abs(), posinf=0)
            if dout is None:
                continue
            g = dout[q0:q1, h]
            dw, dwa = g @ vj.t(), g.abs() @ vj.abs().t()
            delta, da = (w * dw).sum(1, keepdim=True), (g.abs() * out.abs()).sum(1, keepdim=True)
            edelta = (g.abs() * (eo + u * (out.abs() + eo))).sum(1, keepdim=True) + (dim + 2) * F32 * da
            dx = w * (dw - delta)
            edx = ew * (dw - delta).abs() + w * ((dim + 4) * F32 * dwa + edelta)
            edx = edx + u * (dx.abs() + edx)
            ew = ew + u * (w + ew)
            dq = dx @ kj * scale
            eq = (edx @ kj.abs() + (n + 4) * F32 * (dx.abs() @ kj.abs())) * scale
            res["dq"][0][q0:q1, h], res["dq"][1][q0:q1, h] = dq, eq + u * (dq.abs() + eq)
            m = group * (q1 - q0) + 4
            res["dk"][0][k0:k1, c] += dx.t() @ qi * scale
            res["dk"][1][k0:k1, c] += (edx.t() @ qi.abs() + m * F32 * (dx.abs().t() @ qi.abs())) * scale
            res["dv"][0][k0:k1, c] += w.t() @ g
            res["dv"][1][k0:k1, c] += ew.t() @ g.abs() + m * F32 * (w.t() @ g.abs())
    for name in ("dk", "dv") if dout is not None else ():
        value, bound = res[name]
        res[name][1] = bound + u * (value.abs() + bound)
    # float16 results below its normal numbers are rounded to its smallest step
    tiny = torch.finfo(typ).tiny * torch.finfo(typ).eps / 2
    return {n: (x, e + (tiny if n != "lse" else 0)) for n, (x, e) in res.items()}


def cache_rows(pool, table_row, positions):
    """Rows of a pool [P, H, page, D] at a clip's positions: [n, H, D]."""
    page = pool.shape[2]
    return torch.stack([pool[table_row[j // page], :, j % page] for j in positions]) if positions else pool.new_zeros(
        (0, pool.shape[1], pool.shape[3]))


def cache_attention(q, k_pool, v_pool, table, lens, window, sinks, scale):
    """(out, bound) of the newest frames."""
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    k_pool, v_pool, table = k_pool.cpu(), v_pool.cpu(), table.cpu().tolist()
    for b, n in enumerate(lens.tolist()):
        at = [j for j in range(n) if window is None or n - 1 - j < window or j < sinks]
        k, v = cache_rows(k_pool, table[b], at), cache_rows(v_pool, table[b], at)
        one = attention(q[b:b + 1], k, v, [0, 1], [0, len(at)], None, 0, scale)["out"]
        out[b], bound[b] = one[0][0], one[1][0]
    return out, bound


# ---------------------------------------------------------------- pages, one entry after another

def reserve(table, lens, new_lens, refs, page):
    table, refs = [list(r) for r in table], list(refs)
    free, missing = [p for p, n in enumerate(refs) if n <= 0], 0
    for b, row in enumerate(table):
        for e in range(-(-max(lens[b], 0) // page), -(-max(new_lens[b], 0) // page)):
            if e >= len(row) or not free:
                missing += 1
                continue
            row[e] = free.pop(0)
            refs[row[e]] = 1
    return table, refs, missing


def fork(table, lens, refs, parents, children, page, copies):
    """``copies`` gets the (source, target) pairs."""
    old, was = [list(r) for r in table], list(lens)
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    free, missing, pages = [p for p, n in enumerate(refs) if n <= 0], 0, len(refs)
    for parent, child in zip(parents, children):
        if not (0 <= parent < len(old) and 0 <= child < len(old)):
            continue
        for p in old[child]:
            if 0 <= p < pages:
                refs[p] -= 1
        row, n = list(old[parent]), was[parent]
        part = n // page if n % page and n // page < len(row) else None
        for e, p in enumerate(row):
            if e != part and 0 <= p < pages:
                refs[p] += 1
        if part is not None:
            source, row[part] = row[part], -1
            if free:
                row[part] = free.pop(0)
                refs[row[part]] += 1
                copies.append((source, row[part]))
            else:
                missing += 1
        table[child], lens[child] = row, n
    return table, lens, refs, missing


def free(table, lens, refs, page, drop, window, sinks):
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    for b, row in enumerate(table):
        gone = drop is not None and drop[b] != 0
        for e, p in enumerate(row):
            later = any(j < sinks or lens[b] - j < window for j in range(e * page, (e + 1) * page)) if window is not None else True
            if gone or not later:
                if 0 <= p < len(refs):
                    refs[p] -= 1
                row[e] = -1
        if gone:
            lens[b] = 0
    return table, lens, refs


def compact(table, refs, copies):
    live = sum(n > 0 for n in refs)
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    holes = [p for p in range(live) if refs[p] <= 0]
    new = dict(zip(movers, holes))
    copies.extend(new.items())
    table = [[new.get(p, p) for p in row] for row in table]
    out = [0] * len(refs)
    for p, n in enumerate(refs):
        if n > 0:
            out[new.get(p, p)] = n
    return table, out, live
