"""The 64-bit backward of training_reference against central differences of
its forward, with each kind of bias; the forward against the oracle; and the
bucket map against its definition."""
import math

import numpy as np
import pytest

import masked_attention_fa_b200 as fa
import oracle
import training_reference as ref
from oracle import Problem

CASES = [
    (dict(layout="BNSD", B=1, N=2, Sq=5, Skv=7, D=4, sparse_mode=3), {}),
    (dict(layout="BSND", B=2, N=1, Sq=6, Skv=4, D=4, sparse_mode=3), dict(alibi="sqrt")),
    (dict(layout="TND", B=3, N=2, Sq=7, Skv=9, D=4, sparse_mode=0, actual_seq_qlen=[3, 3, 7],
          actual_seq_kvlen=[4, 6, 9]), dict(bias=True)),
    (dict(layout="BNSD", B=1, N=2, Sq=6, Skv=6, D=4, sparse_mode=4, pre_tokens=2, next_tokens=1),
     dict(bias=True)),
]


def _inputs(kw, opt, seed):
    g = np.random.default_rng(seed)
    pb = Problem(**kw)
    q, k, v = (g.standard_normal(s) for s in (pb.q_shape(), pb.kv_shape(), pb.kv_shape()))
    bias = {}
    if "alibi" in opt:
        bias = dict(alibi=opt["alibi"], slopes=g.uniform(0.1, 1, pb.N))
    if "bias" in opt:
        bias = dict(table=g.standard_normal((8, pb.N)), bucket_of=fa.relative_buckets(8, 4))
    return pb, q, k, v, bias, g


@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward_matches_differences(case):
    kw, opt = CASES[case]
    pb, q, k, v, bias, g = _inputs(kw, opt, 50 + case)
    o, lse = ref.forward(pb, q, k, v, **bias)
    do = g.standard_normal(o.shape)
    dl = np.where(np.isinf(lse), 0.0, g.standard_normal(lse.shape))

    def loss():
        oo, ll = ref.forward(pb, q, k, v, **bias)
        return (oo * do).sum() + (np.where(np.isinf(ll), 0.0, ll) * dl).sum()

    got = ref.backward(pb, q, k, v, o, lse, do, dlse=dl, **bias)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dtable", bias.get("table"))):
        if x is None:
            continue
        grad = np.zeros(x.shape)
        for at in np.ndindex(x.shape):
            keep, step = x[at], 1e-5
            x[at] = keep + step
            up = loss()
            x[at] = keep - step
            grad[at] = (up - loss()) / (2 * step)
            x[at] = keep
        np.testing.assert_allclose(got[name][0], grad, rtol=0, atol=1e-8)


@pytest.mark.parametrize("case", [0, 1])
def test_forward_matches_oracle(case):
    kw, opt = CASES[case]
    pb, q, k, v, bias, _ = _inputs(kw, opt, 60 + case)
    o, lse = ref.forward(pb, q, k, v, **bias)
    o2, lse2 = oracle.attention(pb, q, k, v, **bias)
    np.testing.assert_allclose(o, o2, atol=1e-12)
    np.testing.assert_allclose(lse, lse2, atol=1e-12)


@pytest.mark.parametrize("buckets,reach,two_sided", [(32, 128, True), (32, 128, False), (8, 20, True),
                                                     (10, 33, False), (64, 256, True)])
def test_bucket_map(buckets, reach, two_sided):
    m = fa.relative_buckets(buckets, reach, two_sided)
    assert m.dtype == np.int32 and m.shape == (2 * reach + 1,)
    side = buckets // 2 if two_sided else buckets
    single = side // 2
    for rel in range(-reach, reach + 1):
        d = abs(rel) if two_sided else max(-rel, 0)
        base = side if two_sided and rel > 0 else 0
        if d < single:
            assert m[rel + reach] == base + d
        else:
            # the largest step whose start, single * (reach / single)^(n / steps), d has reached
            steps = side - single
            n = max(x for x in range(steps + 1)
                    if d * (1 + 1e-12) >= single * (reach / single) ** (x / steps))
            assert m[rel + reach] == base + min(single + n, side - 1)
    assert m.max() == buckets - 1 and m.min() == 0


def test_bucket_map_refusals():
    with pytest.raises(ValueError):
        fa.relative_buckets(2, 10)
    with pytest.raises(ValueError):
        fa.relative_buckets(32, 8)
    assert math.isclose(fa.relative_buckets(4, 2)[0], 1)
