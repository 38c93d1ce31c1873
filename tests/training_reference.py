"""The training operators in 64 bits, straight from their formulas, for the
tests: the forward with a bias, its backward, and elementwise bounds on what
the kernels' roundings can change. Visibility comes from the oracle's explicit
matrices.

Bounds. The kernels hold every sum, statistic and norm in fp32 and round three
things to bf16 (half a step is u = 2^-8 relative): P and dS, as operands of
the products that sum over them, and each output. With w = 2^-13 for the
relative error of an fp32 P (a score is a sum of D <= 128 products: (D + 2)
2^-24 sum |q||k| scale <= 130 * 2^-24 * 8 = 6.2e-5 for N(0, 1) operands; exp2,
lse and scale add less than 1e-5 more; 2^-13 = 1.2e-4), and with m = |dO||V|^T
+ sum |dO||o| + |dlse| bounding what dP - delta is a difference of (its fp32
error is below 130 * 2^-24 m < w m):
    |d(dv)| <= u |dv| + (u + w) P^T |dO|
    |d(dS)| <= w |dS| + w P m            before it is rounded
    |d(dq)| <= u |dq| + scale ((u + w) |dS| + w P m) |K|     (dk alike)
    |d(dtable)| <= sum over the bucket of w |dS| + w P m
each with (1 + 2^-6) for products of the error terms.
"""
import numpy as np

import oracle

U, W, SLACK = 2.0 ** -8, 2.0 ** -13, 1.0 + 2.0 ** -6


def f64(t):
    return t.detach().cpu().double().numpy()


def heads(x, layout, b, off, n):
    """[N, n, D] view of sequence b's tokens."""
    if layout == "BNSD":
        return x[b]
    if layout == "BSND":
        return x[b].transpose(1, 0, 2)
    return x[off:off + n].transpose(1, 0, 2)


def rows(x, layout, b, off, n):
    return x[:, off:off + n] if layout == "TND" else x[b]


def bias_of(sq, skv, alibi=None, slope=None, table=None, bucket_of=None, h=0):
    """[sq, skv] bias of one head, and the bucket of each pair."""
    rel = np.arange(skv)[None, :] - (np.arange(sq)[:, None] + (skv - sq))
    if alibi is not None:
        if alibi == "left":
            return slope * np.broadcast_to(np.arange(skv, dtype=np.float64), rel.shape), None
        return slope * (np.sign(rel) * np.sqrt(np.abs(rel)) if alibi == "sqrt" else rel), None
    if table is not None:
        R = len(bucket_of) // 2
        bucket = np.asarray(bucket_of)[np.clip(rel, -R, R) + R]
        return table[bucket, h], bucket
    return np.zeros(rel.shape), None


def forward(pb, q, k, v, alibi=None, slopes=None, table=None, bucket_of=None):
    """(o, lse) in 64 bits."""
    o = np.zeros(pb.q_shape())
    lse = np.full(pb.lse_shape(), -np.inf)
    for b in range(pb.B):
        qo, ko, sq, skv = pb.seq(b)
        if sq == 0 or skv == 0:
            continue
        Q, K, V = (heads(x, pb.layout, b, f, n) for x, f, n in
                   ((q, qo, sq), (k, ko, skv), (v, ko, skv)))
        for h in range(pb.N):
            see = oracle.mask_matrix(pb, b, h) != 0
            bias, _ = bias_of(sq, skv, alibi, None if slopes is None else slopes[h], table,
                              bucket_of, h)
            s = np.where(see, Q[h] @ K[h].T * pb.scale + bias, -np.inf)
            top = np.where(see.any(1), s.max(1), 0.0)
            e = np.exp(s - top[:, None])
            den = e.sum(1)
            heads(o, pb.layout, b, qo, sq)[h] = (e @ V[h]) / np.where(den > 0, den, 1)[:, None]
            with np.errstate(divide="ignore"):
                rows(lse, pb.layout, b, qo, sq)[h] = np.log(den) + top
    return o, lse


def backward(pb, q, k, v, o, lse, do, dlse=None, alibi=None, slopes=None, table=None,
             bucket_of=None):
    """{"dq", "dk", "dv"[, "dtable"]} -> (value, bound on a kernel's error)."""
    out = {n: [np.zeros(s), np.zeros(s)] for n, s in
           (("dq", pb.q_shape()), ("dk", pb.kv_shape()), ("dv", pb.kv_shape()))}
    if table is not None:
        out["dtable"] = [np.zeros(table.shape), np.zeros(table.shape)]
    for b in range(pb.B):
        qo, ko, sq, skv = pb.seq(b)
        if sq == 0 or skv == 0:
            continue
        Q, O, G = (heads(x, pb.layout, b, qo, sq) for x in (q, o, do))
        K, V = (heads(x, pb.layout, b, ko, skv) for x in (k, v))
        L = rows(lse, pb.layout, b, qo, sq)
        for h in range(pb.N):
            see = oracle.mask_matrix(pb, b, h) != 0
            bias, bucket = bias_of(sq, skv, alibi, None if slopes is None else slopes[h], table,
                                   bucket_of, h)
            live = np.where(np.isinf(L[h]), 0.0, L[h])
            p = np.where(see, np.exp(Q[h] @ K[h].T * pb.scale + bias - live[:, None]), 0.0)
            delta = (G[h] * O[h]).sum(1)
            m = np.abs(G[h]) @ np.abs(V[h]).T + (np.abs(G[h]) * np.abs(O[h])).sum(1)[:, None]
            if dlse is not None:
                dl = rows(dlse, pb.layout, b, qo, sq)[h]
                delta, m = delta - dl, m + np.abs(dl)[:, None]
            ds = p * (G[h] @ V[h].T - delta[:, None])
            eds = W * np.abs(ds) + W * p * m
            er = eds + U * np.abs(ds)

            def put(name, first, n, value, err):
                heads(out[name][0], pb.layout, b, first, n)[h] = value
                heads(out[name][1], pb.layout, b, first, n)[h] = SLACK * (U * np.abs(value) + err)

            put("dq", qo, sq, pb.scale * ds @ K[h], pb.scale * er @ np.abs(K[h]))
            put("dk", ko, skv, pb.scale * ds.T @ Q[h], pb.scale * er.T @ np.abs(Q[h]))
            put("dv", ko, skv, p.T @ G[h], (U + W) * p.T @ np.abs(G[h]))
            if table is not None:
                for c in range(table.shape[0]):
                    out["dtable"][0][c, h] += ds[bucket == c].sum()
                    out["dtable"][1][c, h] += SLACK * eds[bucket == c].sum()
    return {n: tuple(x) for n, x in out.items()}


def check(got, ref, what=""):
    """Every element inside its bound (2^-120 for elements whose bound is 0 or underflows)."""
    for name, g in zip(ref, got):
        value, bound = ref[name]
        g = f64(g)
        assert g.shape == value.shape, f"{what} {name}"
        assert np.isfinite(g).all(), f"{what} {name}: non-finite"
        excess = np.abs(g - value) - bound - 2.0 ** -120
        at = np.unravel_index(excess.argmax(), excess.shape) if excess.size else ()
        assert excess.size == 0 or excess.max() <= 0, (
            f"{what} {name}{at}: {g[at]} against {value[at]}, bound {bound[at]}")
