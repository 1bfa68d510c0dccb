"""A block's norms, routing and experts from their definitions, in 64 bits on the host, with bounds on what the
kernels' roundings can come to."""
import math

import numpy as np
import torch

U = 2.0 ** -24     # fp32: half a step, relative
B = 2.0 ** -8      # bf16


def norm(u, r, post, gate, pre, alpha, beta, offset, eps):
    """r', h and the bounds of their errors before they are rounded.  u, r [T, D]; gate [rows, D] or None."""
    u, r = u.double(), r.double()
    t = u.shape[0]
    n = u
    if post is not None:
        n = u / torch.sqrt(u.pow(2).mean(1, keepdim=True) + eps) * (post.double() + offset)
    if gate is not None:
        n = n * gate.double().repeat_interleave(t // gate.shape[0], 0)
    res = alpha * r + beta * n
    # a mean square: at most 16 + 10 additions one behind another, a square and a division; its root halves that.
    # Then the root, the reciprocal and up to four products: 13 + 2 + 6 roundings, taken as 32.
    err = 32 * U * (abs(alpha) * r.abs() + abs(beta) * n.abs())
    if pre is None:
        return res, err, None, None
    f = 1 / torch.sqrt(res.pow(2).mean(1, keepdim=True) + eps)
    w = pre.double() + offset
    h = res * f * w
    # the error of r' moves the mean square by at most its own share of the norm
    moved = err.pow(2).mean(1, keepdim=True).sqrt() * f
    return res, err, h, (err * f + res.abs() * f * (moved + 32 * U)) * w.abs()


def route(logits, cfg, bias=None, live=None):
    """ids [T, k] and weights [T, k] (float64) of logits [T, E] (float64 numpy)."""
    t, e = logits.shape
    k, groups = cfg["k"], cfg.get("groups", 1)
    size, tops, best = e // groups, cfg.get("top_groups", 1), cfg.get("group_best", 1)
    ids, weights = np.full((t, k), -1, dtype=np.int64), np.zeros((t, k))
    b = np.zeros(e) if bias is None else np.asarray(bias, dtype=np.float64)
    for row in range(t if live is None else max(0, min(t, live))):
        l = logits[row]
        softmax = cfg.get("score", 0) == 0
        bad = np.isnan(l) | (softmax & (l == np.inf))
        ok = ~bad & (l != -np.inf)
        with np.errstate(over="ignore", invalid="ignore"):
            if softmax:
                if (softmax and (l == np.inf).any()):
                    s = np.zeros(e)
                else:
                    top = l[ok].max() if ok.any() else 0.0
                    z = np.where(ok, np.exp(np.where(ok, l - top, 0.0)), 0.0)
                    s = z / z.sum() if ok.any() else z
            else:
                s = np.where(ok, 1 / (1 + np.exp(-np.where(ok, l, 0.0))), 0.0)
        c = np.where(bad, np.inf, np.where(ok, s + b if bias is not None else l, -np.inf))   # without a bias: the logits' order
        kept = np.ones(e, dtype=bool)
        if groups > 1:
            v = np.where(bad, np.inf, np.where(ok, s + b, -np.inf)).reshape(groups, size)
            order = -np.sort(-v, axis=1)
            score = order[:, 0] if best == 1 else np.where(order[:, 1] == -np.inf, -np.inf, order[:, 0] + order[:, 1])
            if best == 1 and bias is None:
                score = np.where(bad, np.inf, l).reshape(groups, size).max(1)
            chosen = sorted(range(groups), key=lambda g: (-score[g], g))[:tops]
            kept = np.repeat(np.isin(np.arange(groups), chosen), size)
        pool = [i for i in range(e) if kept[i] and c[i] > -np.inf]
        pool = sorted(pool, key=lambda i: (-c[i], i))[:k]
        ids[row, : len(pool)] = pool
        x = l[pool]
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            if not cfg.get("renormalise", True):
                w = s[pool]
            elif softmax:
                w = np.exp(x - x.max()) if len(pool) else x
                w = w / w.sum()
            else:   # log s, so that very negative logits keep their ratio
                ls = -np.logaddexp(0.0, -x)
                w = np.exp(ls - ls.max()) if len(pool) else x
                w = w / w.sum()
        weights[row, : len(pool)] = np.nan if bad.any() else w * cfg.get("scale", 1.0)
    return ids, weights


def experts(x, ids, weights, gate_up, down):
    """y [T, H] and its bound: x [T, H], gate_up [E, 2 I, H] and down [E, H, I] as the values they stand for."""
    x = x.double()
    t, h = x.shape
    inner = down.shape[2]
    y, var, lin = (torch.zeros((t, h), dtype=torch.float64) for _ in range(3))
    # a sum of K products: 128 of a group in the matrix unit (which may cut instead of round: a whole step each), then
    # the group's scale, the groups one behind another and the warps' sums
    steps = lambda n: (128 + n // 128 + 16) * 2 * U  # noqa: E731

    # a bf16 is held as two e4m3 under the power of two of the largest in its group of 128: exact down to 2^-13 of that power of
    # two, below it off by half a step of the first (2^-10 of 2^7) and of the second (a sixteenth of that)
    def lost(v):
        top = v.abs().reshape(-1, 128).amax(1, keepdim=True).expand(-1, 128).reshape(-1)
        return torch.where(v.abs() < 2.0 ** -12 * top, 2.0 ** -17 * (17 / 16) * top, 0.0)

    for row in range(t):
        for j in range(ids.shape[1]):
            e = int(ids[row, j])
            if e < 0 or e >= gate_up.shape[0]:
                continue
            g, u = (gate_up[e] @ x[row]).split(inner)
            lg, lu = (gate_up[e].abs() @ lost(x[row])).split(inner)
            ag, au = (gate_up[e].abs() @ x[row].abs()).split(inner)
            s = g * torch.sigmoid(g)
            hid = s * u
            # |silu'| <= 1.1
            e_hid = 1.1 * (steps(h) * ag + lg) * u.abs() + s.abs() * (steps(h) * au + lu) + 8 * U * hid.abs()
            w = float(weights[row, j])
            y[row] += w * (down[e] @ hid)
            lin[row] += abs(w) * (down[e].abs() @ (e_hid + steps(inner) * hid.abs() + lost(hid)))
            var[row] += w * w * (down[e].pow(2) @ hid.pow(2))
    # each h is rounded by at most B relative, evenly spread: a standard deviation of B / sqrt(3); six of them
    return y, lin + 6 * B / math.sqrt(3) * var.sqrt() + 40 * U * y.abs()


def close(got, want, bound, rounding):
    """got within bound of want, and within one rounding of that."""
    got = got.double().cpu()
    err = (got - want).abs()
    limit = bound + rounding * (want.abs() + bound) + 1e-37
    bad = ~(err <= limit)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist(), limit[bad][:3].tolist())
