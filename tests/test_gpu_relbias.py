"""The learned relative position bias: its forward against the 64-bit
formulas, its backward with the table's gradient inside the bounds derived in
training_reference, on every closed-form mode and layout; distances below,
inside and beyond the reach in one tile; bucket maps that are not monotone;
the chain of both; equal bits on a second call; and the refusals."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import assert_close, problem_of
from masked_attention_fa_b200.workloads import random_inputs
from test_gpu_backward import CASES, args_of

pytestmark = pytest.mark.gpu

CLOSED = sorted(n for n in CASES if not n.startswith("mask"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def maps(seed, kind):
    """A bucket map and its number of buckets."""
    if kind == "log":
        return fa.relative_buckets(32, 128), 32
    if kind == "one_sided":
        return fa.relative_buckets(10, 33, False), 10
    g = np.random.default_rng(seed)
    reach, buckets = {"shuffled": (70, 9), "tiny": (1, 3), "wide": (500, 320)}[kind]
    return g.integers(0, buckets, 2 * reach + 1).astype(np.int32), buckets


def setup(name, D, kind, seed):
    c = dict(CASES[name], D=D)
    lens = {k: c.pop(k) for k in ("prefix", "cu_q", "cu_kv") if k in c}
    inp = random_inputs(c["layout"], c["B"], c["N"], c["Sq"], c["Skv"], D, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    m, buckets = maps(seed, kind)
    table = torch.randn(buckets, c["N"], generator=g)
    do = torch.randn(inp["q"].shape, generator=g).to(torch.bfloat16)
    pb = problem_of(c, None, lens.get("prefix"), lens.get("cu_q"), lens.get("cu_kv"))
    return c, lens, inp, m, table, do, pb


def gpu(inp):
    return [inp[x].cuda() for x in "qkv"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["log", "one_sided", "shuffled"])
@pytest.mark.parametrize("name", CLOSED)
def test_forward(name, kind, D):
    c, lens, inp, m, table, _, pb = setup(name, D, kind, 5000)
    attn = fa.MaskedAttention(**c)
    o, lse = attn(*gpu(inp), rel_bias=table.cuda(), rel_buckets=m, **args_of(lens))
    attn.sync_status()
    attn.close()
    want = ref.forward(pb, *(ref.f64(inp[x]) for x in "qkv"), table=ref.f64(table), bucket_of=m)
    assert_close(ref.f64(o.float()), ref.f64(lse), *want, f"{name} {kind}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["log", "one_sided", "shuffled", "tiny", "wide"])
@pytest.mark.parametrize("name", CLOSED)
def test_backward(name, kind, D):
    c, lens, inp, m, table, do, pb = setup(name, D, kind, 5100)
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    o, lse = ref.forward(pb, q, k, v, table=ref.f64(table), bucket_of=m)
    o, lse = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()
    want = ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do), table=ref.f64(table),
                        bucket_of=m)
    attn = fa.MaskedAttention(**c)
    got = attn.backward(do.cuda(), *gpu(inp), o.cuda(), lse.cuda(), rel_bias=table.cuda(),
                        rel_buckets=m, **args_of(lens))
    attn.sync_status()
    attn.close()
    ref.check(got, want, f"{name} {kind}")


def test_training_step_of_one_handle():
    """Forward and backward in turn on one handle, the table changing between
    the steps and the bucket map once; equal bits when a step is repeated."""
    c, lens, inp, m, table, do, pb = setup("rightdown", 128, "log", 5200)
    attn = fa.MaskedAttention(**c)
    q, k, v = gpu(inp)
    seen = []
    for step, (mm, t) in enumerate([(m, table), (m, table * 2), (maps(3, "shuffled")[0], table),
                                    (m, table)]):
        t = t.cuda()
        o, lse = attn(q, k, v, rel_bias=t, rel_buckets=mm)
        got = attn.backward(do.cuda(), q, k, v, o, lse, rel_bias=t, rel_buckets=mm)
        want = ref.backward(pb, *(ref.f64(inp[x]) for x in "qkv"), ref.f64(o), ref.f64(lse),
                            ref.f64(do), table=ref.f64(t), bucket_of=mm)
        ref.check(got, want, f"step {step}")
        seen.append((o, lse, *got))
    attn.sync_status()
    for a, b in zip(seen[0], seen[3]):
        assert torch.equal(a, b)
    # a plain call of the same handle is the plain operator
    plain = fa.MaskedAttention(**c)
    for a, b in zip(attn(q, k, v), plain(q, k, v)):
        assert torch.equal(a, b)
    attn.close()
    plain.close()


def test_claimed_work():
    """1,300 packed sequences x 2 heads: enough items to claim at run time."""
    g = torch.Generator().manual_seed(5300)
    lens = torch.randint(1, 260, (1300,), generator=g)
    cu = torch.cumsum(lens, 0).tolist()
    c = dict(layout="TND", B=1300, N=2, Sq=cu[-1], Skv=cu[-1], D=128, sparse_mode=3)
    inp = random_inputs("TND", 1300, 2, cu[-1], cu[-1], 128, seed=5301)
    m, buckets = maps(0, "log")
    table = torch.randn(buckets, 2, generator=g)
    do = torch.randn(cu[-1], 2, 128, generator=g).to(torch.bfloat16)
    pb = problem_of(c, None, None, cu, cu)
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    a = dict(rel_bias=table.cuda(), rel_buckets=m, actual_seq_qlen=cu, actual_seq_kvlen=cu)
    attn = fa.MaskedAttention(**c)
    o, lse = attn(*gpu(inp), **a)
    got = attn.backward(do.cuda(), *gpu(inp), o, lse, **a)
    attn.sync_status()
    attn.close()
    assert_close(ref.f64(o.float()), ref.f64(lse),
                 *ref.forward(pb, q, k, v, table=ref.f64(table), bucket_of=m), "claimed")
    ref.check(got, ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do),
                                table=ref.f64(table), bucket_of=m), "claimed")


def test_refusals():
    c, lens, inp, m, table, do, pb = setup("causal", 64, "log", 5400)
    attn = fa.MaskedAttention(**c)
    q, k, v = gpu(inp)
    t = table.cuda()
    o = torch.full_like(q, 3.0)
    for bad in (dict(rel_bias=t), dict(rel_bias=t.half(), rel_buckets=m),
                dict(rel_bias=t[:, :-1], rel_buckets=m), dict(rel_bias=t.cpu(), rel_buckets=m),
                dict(rel_bias=t, rel_buckets=m[:-1]),
                dict(rel_bias=t, rel_buckets=m, slopes=torch.ones(c["N"], device="cuda"))):
        with pytest.raises(ValueError):
            attn(q, k, v, out=o, **bad)
    for bad_map, status in ((m + 1, "FA_ERR_PARAM_INVALID"), (m - 1, "FA_ERR_PARAM_INVALID"),
                            (np.zeros(2051, np.int32), "FA_ERR_UNSUPPORTED")):
        with pytest.raises(fa.FaError) as e:
            attn(q, k, v, out=o, rel_bias=t, rel_buckets=bad_map)
        assert e.value.name == status
    with pytest.raises(fa.FaError) as e:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            attn(q, k, v, out=o, rel_bias=t, rel_buckets=m)
    assert e.value.name == "FA_ERR_UNSUPPORTED"
    torch.cuda.synchronize()
    assert (o == 3.0).all()
    attn.close()
    for kw, status in ((dict(alibi="right"), "FA_ERR_PARAM_INVALID"),
                       (dict(sparse_mode=1, mask_kind="SS"), "FA_ERR_UNSUPPORTED")):
        a = fa.MaskedAttention(**dict(c, **kw))
        with pytest.raises(fa.FaError) as e:
            a(q, k, v, rel_bias=t, rel_buckets=m)
        assert e.value.name == status
        a.close()
