"""The backward pass where dS is written to memory (head dim 128, more than 4
work items per SM), against its formulas in 64 bits inside the bounds derived
in training_reference: packed sequences of every length around the tile, dense
masks, ALiBi, the learned bias; dS held in several shares; sequences whose
neighbours hold NaN; equal bits on a second call and against a call whose dS
does not fit."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import problem_of
from masked_attention_fa_b200.workloads import alibi_slopes, block_mask, random_inputs

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def packed(mode, n, seed, N=2, **extra):
    g = np.random.default_rng(seed)
    lens_q = g.choice([0, 1, 2, 127, 128, 129, 200, 257, 300], n)
    lens_kv = np.where(g.random(n) < 0.5, lens_q, g.choice([0, 1, 64, 128, 130, 255, 256, 310], n))
    cu_q, cu_kv = np.cumsum(lens_q).tolist(), np.cumsum(lens_kv).tolist()
    c = dict(layout="TND", sparse_mode=mode, B=n, N=N, Sq=cu_q[-1], Skv=cu_kv[-1], D=D, **extra)
    return c, dict(cu_q=cu_q, cu_kv=cu_kv)


CASES = {
    "packed": lambda: packed(3, 230, 1),
    "packed_all": lambda: packed(0, 230, 2),
    "packed_band": lambda: packed(4, 230, 3, pre_tokens=90, next_tokens=40),
    "causal": lambda: (dict(layout="BNSD", sparse_mode=2, B=2, N=50, Sq=390, Skv=390, D=D), {}),
    "rightdown_dead_rows": lambda: (dict(layout="BSND", sparse_mode=3, B=1, N=80, Sq=515, Skv=390, D=D), {}),
    "prefix": lambda: (dict(layout="BNSD", sparse_mode=5, B=2, N=50, Sq=300, Skv=510, D=D),
                       dict(prefix=[0, 400])),
    "mask_bnss": lambda: (dict(layout="BNSD", sparse_mode=1, B=2, N=50, Sq=390, Skv=300, D=D,
                               mask_kind="BNSS"), {}),
    "mask_b1ss": lambda: (dict(layout="BSND", sparse_mode=1, B=2, N=50, Sq=300, Skv=390, D=D,
                               mask_kind="B1SS"), {}),
}


def setup(name, bias=None, seed=6000):
    c, lens = CASES[name]()
    tiles = lambda lens_: sum((int(x) + 127) // 128 for x in lens_)
    if c["layout"] == "TND":
        items = tiles(np.diff([0] + lens["cu_q"])) + tiles(np.diff([0] + lens["cu_kv"]))
    else:
        items = c["B"] * (tiles([c["Sq"]]) + tiles([c["Skv"]]))
    assert items * c["N"] > 4 * 148, "the case does not reach the path under test"
    inp = random_inputs(c["layout"], c["B"], c["N"], c["Sq"], c["Skv"], D, seed=seed)
    mask = None
    if c.get("mask_kind"):
        shape = {"B1SS": (c["B"], 1), "BNSS": (c["B"], c["N"])}[c["mask_kind"]]
        mask = block_mask(shape + (c["Sq"], c["Skv"]), seed=seed)
        mask[..., c["Sq"] // 3, :] = 1
    g = torch.Generator().manual_seed(seed + 1)
    kw, call = {}, {}
    if bias == "right":
        kw = dict(alibi="right", slopes=np.array(alibi_slopes(c["N"]), dtype=np.float64))
        call = dict(slopes=torch.tensor(kw["slopes"], dtype=torch.float32, device="cuda"))
    elif bias == "learned":
        table = torch.randn(20, c["N"], generator=g)
        m = fa.relative_buckets(20, 90)
        kw = dict(table=ref.f64(table), bucket_of=m)
        call = dict(rel_bias=table.cuda(), rel_buckets=m)
    pb = problem_of(c, mask, lens.get("prefix"), lens.get("cu_q"), lens.get("cu_kv"))
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    o, lse = ref.forward(pb, q, k, v, **kw)
    o, lse = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()
    do = torch.randn(o.shape, generator=g).to(torch.bfloat16)
    want = ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do), **kw)
    t = dict(do=do, q=inp["q"], k=inp["k"], v=inp["v"], o=o, lse=lse)
    return c, lens, mask, t, want, call


def run(c, lens, mask, t, call, attn=None):
    own = attn is None
    attn = attn or fa.MaskedAttention(**c, alibi="right" if "slopes" in call else None)
    got = attn.backward(*(x.cuda() for x in t.values()), atten_mask=None if mask is None else mask.cuda(),
                        prefix=lens.get("prefix"), actual_seq_qlen=lens.get("cu_q"),
                        actual_seq_kvlen=lens.get("cu_kv"), **call)
    torch.cuda.synchronize()
    attn.sync_status()
    if own:
        attn.close()
    return got


@pytest.mark.parametrize("bias", [None, "right", "learned"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_formula(name, bias):
    if bias and name.startswith("mask"):
        pytest.skip("a mask goes with no bias")
    c, lens, mask, t, want, call = setup(name, bias)
    ref.check(run(c, lens, mask, t, call), want, name)


@pytest.mark.parametrize("name,bias", [("packed", None), ("mask_bnss", None), ("prefix", "learned")])
def test_shares(name, bias, monkeypatch):
    """The same bits with dS in one share, in shares of at most 20 tiles (two
    or three heads each), and (but for dq, a sum in another order of products)
    with no room for it at all."""
    c, lens, mask, t, want, call = setup(name, bias)
    whole = run(c, lens, mask, t, call)
    again = run(c, lens, mask, t, call)
    monkeypatch.setenv("FA_TEST_SPILL_TILES", "20")
    shares = run(c, lens, mask, t, call)
    monkeypatch.setenv("FA_TEST_SPILL_TILES", "1")
    walks = run(c, lens, mask, t, call)
    for x, y, z in zip(whole, again, shares):
        assert torch.equal(x, y) and torch.equal(x, z)
    for x, y in zip(whole[1:], walks[1:]):
        assert torch.equal(x, y)
    ref.check(walks, want, name)


def test_nan_of_another_sequence_stays_there():
    c, lens, mask, t, want, call = setup("packed")
    cu_q, cu_kv = [0] + lens["cu_q"], [0] + lens["cu_kv"]
    t = {n: x.clone() for n, x in t.items()}
    bad = range(5, c["B"], 7)
    for b in bad:
        for n in ("do", "q", "o"):
            t[n][cu_q[b]:cu_q[b + 1]] = float("nan")
        for n in ("k", "v"):
            t[n][cu_kv[b]:cu_kv[b + 1]] = float("inf")
    got = run(c, lens, mask, t, call)
    for x, (name, cu) in zip(got, (("dq", cu_q), ("dk", cu_kv), ("dv", cu_kv))):
        x = x.clone()
        value, bound = (y.copy() for y in want[name])
        for b in bad:
            x[cu[b]:cu[b + 1]] = 0
            value[cu[b]:cu[b + 1]] = bound[cu[b]:cu[b + 1]] = 0
        ref.check([x], {name: (value, bound)}, "neighbours")


def test_one_handle_with_and_without():
    """Lengths that take either path in turn on one handle."""
    c, lens, mask, t, want, call = setup("packed")
    attn = fa.MaskedAttention(**c)
    small = [c["Sq"]] * c["B"], [c["Skv"]] * c["B"]  # one sequence takes every token
    first = run(c, lens, mask, t, call, attn)
    run(dict(c), dict(cu_q=small[0], cu_kv=small[1]), mask, t, call, attn)
    for x, y in zip(first, run(c, lens, mask, t, call, attn)):
        assert torch.equal(x, y)
    attn.close()
