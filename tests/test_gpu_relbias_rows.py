"""The forward with the learned relative position bias for sequences of a few
query rows, against its formula in 64 bits.

Bounds. Every sum and statistic is fp32: a score is a sum of D <= 128 products
(error below 130 * 2^-24 * sum |q||k| scale <= 6.2e-5 for N(0, 1) operands),
the bias and the exponential add less than 1e-5, so a weight is off by at most
w = 2^-13 relative and the normalised output by 2 w sum P|v|, and by one
rounding to bf16, 2^-8 |o|; lse by w and two roundings of its own size."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import problem_of
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu
U, W = 2.0 ** -8, 2.0 ** -13


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def dense(layout, mode, B, N, sq, skv, **extra):
    return dict(layout=layout, sparse_mode=mode, B=B, N=N, Sq=sq, Skv=skv, **extra)


def packed(mode, lens_q, lens_kv, N, **extra):
    cu_q, cu_kv = np.cumsum(lens_q).tolist(), np.cumsum(lens_kv).tolist()
    return dict(layout="TND", sparse_mode=mode, B=len(lens_q), N=N, Sq=cu_q[-1], Skv=cu_kv[-1],
                cu_q=cu_q, cu_kv=cu_kv, **extra)


CASES = {
    "one_key": dense("BNSD", 0, 1, 1, 1, 1),
    "one_row_short": dense("BSND", 3, 2, 3, 1, 5),
    "one_row": dense("BSND", 3, 2, 3, 1, 1500),
    "one_row_heads_outer": dense("BNSD", 3, 3, 5, 1, 257),
    "three_rows": dense("BNSD", 3, 2, 2, 3, 2049),
    "four_rows_all": dense("BSND", 0, 1, 4, 4, 700),
    "five_rows": dense("BSND", 3, 1, 2, 5, 700),  # the other path's smallest
    "leftup": dense("BNSD", 2, 1, 2, 4, 900),
    "band_dead_rows": dense("BSND", 4, 1, 2, 4, 600, pre_tokens=-598, next_tokens=600),
    "rows_past_the_keys": dense("BNSD", 3, 1, 2, 4, 2),
    "prefix": dense("BNSD", 5, 2, 2, 2, 513, prefix=[0, 300]),
    "many_heads": dense("BSND", 3, 4, 40, 1, 130),
    "packed": packed(3, [1, 0, 4, 2, 1, 3], [700, 5, 4, 1, 0, 1030], 3),
    "packed_band": packed(4, [2, 1, 4], [600, 20, 300], 2, pre_tokens=100, next_tokens=-1),
}


def setup(name, D, seed, reach=40, table_scale=1.0):
    c = dict(CASES[name], D=D)
    lens = {k: c.pop(k) for k in ("prefix", "cu_q", "cu_kv") if k in c}
    inp = random_inputs(c["layout"], c["B"], c["N"], c["Sq"], c["Skv"], D, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    m = torch.randint(0, 11, (2 * reach + 1,), generator=g).numpy().astype(np.int32)
    table = torch.randn(11, c["N"], generator=g) * table_scale
    pb = problem_of(c, None, lens.get("prefix"), lens.get("cu_q"), lens.get("cu_kv"))
    return c, lens, inp, m, table, pb


def run(c, lens, inp, m, table, attn=None, **extra):
    own = attn is None
    attn = attn or fa.MaskedAttention(**c)
    o, lse = attn(*(inp[x].cuda() for x in "qkv"), rel_bias=table.cuda(), rel_buckets=m,
                  prefix=lens.get("prefix"), actual_seq_qlen=lens.get("cu_q"),
                  actual_seq_kvlen=lens.get("cu_kv"), **extra)
    torch.cuda.synchronize()
    attn.sync_status()
    if own:
        attn.close()
    return o, lse


def check(got, pb, inp, m, table, u=U, w=W):
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    kw = dict(table=ref.f64(table), bucket_of=m)
    o, lse = ref.forward(pb, q, k, v, **kw)
    spread, _ = ref.forward(pb, q, k, np.abs(v), **kw)
    assert (np.abs(ref.f64(got[0]) - o) <= 1.02 * (u * np.abs(o) + 2 * w * spread) + 2.0 ** -120).all()
    dead = np.isneginf(lse)
    assert np.array_equal(dead, np.isneginf(ref.f64(got[1])))
    live = ~dead
    a, b = ref.f64(got[1])[live], lse[live]
    assert (np.abs(a - b) <= w + 2.0 ** -22 * np.abs(b)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_formula(name, D):
    c, lens, inp, m, table, pb = setup(name, D, 7000)
    got = run(c, lens, inp, m, table)
    if name == "five_rows":  # P is rounded to bf16 for the tensor cores
        check(got, pb, inp, m, table, w=U / 2 + W)
    else:
        check(got, pb, inp, m, table)


@pytest.mark.parametrize("reach", [1, 1024])
def test_reaches(reach):
    c, lens, inp, m, table, pb = setup("one_row", 128, 7100, reach=reach)
    check(run(c, lens, inp, m, table), pb, inp, m, table)


def test_large_biases():
    """Biases of hundreds: the maximum moves far between keys."""
    c, lens, inp, m, table, pb = setup("three_rows", 64, 7200, table_scale=200.0)
    got = run(c, lens, inp, m, table)
    check(got, pb, inp, m, table, w=W + 700 * 2.0 ** -23)  # a score of up to 700, rounded


def test_what_is_hidden_does_not_count():
    """NaN and infinities in keys that no row sees, and in other sequences."""
    c, lens, inp, m, table, pb = setup("packed_band", 128, 7300)
    want = run(c, lens, inp, m, table)
    dirty = {n: inp[n].clone() for n in "qkv"}
    dirty["k"][:400], dirty["v"][:400] = float("nan"), float("inf")  # 600 - 100 - 1 .. is visible
    for a, b in zip(run(c, lens, dirty, m, table), want):
        assert torch.equal(a, b)


def test_equal_bits_and_shared_workspace():
    """Repeats, another stream, and calls of other lengths on one handle."""
    c, lens, inp, m, table, _ = setup("one_row", 128, 7400)
    attn = fa.MaskedAttention(**c)
    first = run(c, lens, inp, m, table, attn)
    side = torch.cuda.Stream()
    for _ in range(3):
        for s in (None, side):
            for x, y in zip(first, run(c, lens, inp, m, table, attn, stream=s)):
                assert torch.equal(x, y)
    attn.close()
    c, lens, inp, m, table, pb = setup("packed", 64, 7500)
    attn = fa.MaskedAttention(**c)
    first = run(c, lens, inp, m, table, attn)
    T, S = c["Sq"], c["Skv"]
    run(c, dict(cu_q=[T] * 6, cu_kv=[S] * 6), inp, m, table, attn)  # 11 rows: the other path
    for x, y in zip(first, run(c, lens, inp, m, table, attn)):
        assert torch.equal(x, y)
    attn.close()


def test_decoding_steps_follow_the_full_forward():
    """A prompt's forward, then single tokens against the growing key axis,
    each with its gradient: the rows of one forward over everything."""
    N, D, S, P = 3, 64, 200, 190
    g = torch.Generator().manual_seed(7600)
    q, k, v = (torch.randn(1, S, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    m = fa.relative_buckets(16, 60, bidirectional=False)
    table = torch.randn(16, N, generator=g).cuda()
    full = fa.MaskedAttention("BSND", 1, N, S, S, D, 3)
    o, lse = full(q, k, v, rel_bias=table, rel_buckets=m)
    for t in range(P, S):
        step = fa.MaskedAttention("BSND", 1, N, 1, t + 1, D, 3)
        a = [x[:, y:t + 1].contiguous() for x, y in ((q, t), (k, 0), (v, 0))]
        o1, l1 = step(*a, rel_bias=table, rel_buckets=m)
        assert (o1.float() - o[:, t:t + 1].float()).abs().max() <= 3e-2
        assert (l1 - lse[:, :, t:t + 1]).abs().max() <= 1e-3
        got = step.backward(torch.ones_like(o1), *a, o1, l1, rel_bias=table, rel_buckets=m)
        assert all(torch.isfinite(x).all() for x in got)
        step.close()
    full.close()
