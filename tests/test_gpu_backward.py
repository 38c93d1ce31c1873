"""The backward pass (fa_bwd, fa_bwd_alibi) against its formulas in 64 bits,
element by element inside the bounds derived in training_reference: every
sparse mode, layout and mask kind, head dims 64 and 128, lengths of zero and
one, sizes around the 128-row tile, rows that see nothing, the gradient of
lse; the chain forward -> backward; equal bits on a second call; and the
refusals."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import oracle
import training_reference as ref
from gpu_helpers import problem_of
from masked_attention_fa_b200.workloads import alibi_slopes, block_mask, random_inputs

pytestmark = pytest.mark.gpu


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


# The lens, prefix and mask entries are the calls' arguments, the rest the descriptor's.
CASES = {
    "one_pair": dense("BNSD", 0, 1, 1, 1, 1),
    "one_row": dense("BSND", 3, 2, 3, 1, 333),
    "one_key": dense("BNSD", 0, 1, 2, 300, 1),
    "all": dense("BNSD", 0, 2, 2, 300, 333),
    "tile": dense("BNSD", 0, 1, 2, 128, 128),
    "causal": dense("BNSD", 2, 2, 3, 333, 333),
    "causal_tiles": dense("BSND", 2, 1, 2, 640, 640),
    "leftup_short_rows": dense("BSND", 2, 1, 2, 100, 400),
    "leftup_long_rows": dense("BNSD", 2, 1, 2, 400, 100),
    "rightdown": dense("BSND", 3, 2, 2, 200, 515),
    "rightdown_dead_rows": dense("BNSD", 3, 1, 2, 515, 200),
    "band": dense("BNSD", 4, 1, 3, 400, 700, pre_tokens=90, next_tokens=37),
    "band_left_of_diagonal": dense("BSND", 4, 1, 2, 400, 390, pre_tokens=200, next_tokens=-60),
    "prefix": dense("BNSD", 5, 3, 2, 300, 333, prefix=[0, 40, 333]),
    "prefix_dead_rows": dense("BSND", 6, 2, 2, 400, 150, prefix=[0, 130]),
    "packed": packed(3, [130, 0, 257, 5, 1], [140, 3, 300, 5, 1], 3),
    "packed_all": packed(0, [1, 128, 129, 0], [64, 0, 128, 127], 2),
    "packed_band": packed(4, [200, 64, 300], [210, 500, 100], 2, pre_tokens=100, next_tokens=20),
    "packed_split7": packed(7, [100, 200, 0], [120, 260, 7], 2, pre_tokens=300, next_tokens=-40),
    "packed_split8": packed(8, [0, 150, 300], [3, 190, 350], 2, pre_tokens=200, next_tokens=10),
    "mask_ss": dense("BNSD", 1, 2, 2, 300, 333, mask_kind="SS"),
    "mask_b1ss": dense("BSND", 1, 2, 3, 257, 384, mask_kind="B1SS"),
    "mask_bnss": dense("BNSD", 1, 2, 2, 384, 200, mask_kind="BNSS"),
    "mask_band": dense("BNSD", 0, 1, 2, 400, 400, mask_kind="SS", pre_tokens=150, next_tokens=30),
    "mask_aligned": dense("BNSD", 1, 1, 2, 512, 640, mask_kind="SS"),
}


def setup(name, D, seed, alibi=None, with_dlse=False):
    c = dict(CASES[name], D=D)
    lens = {k: c.pop(k) for k in ("prefix", "cu_q", "cu_kv") if k in c}
    inp = random_inputs(c["layout"], c["B"], c["N"], c["Sq"], c["Skv"], D, seed=seed)
    mask = None
    if c.get("mask_kind"):
        shape = {"SS": (), "B1SS": (c["B"], 1), "BNSS": (c["B"], c["N"])}[c["mask_kind"]]
        mask = block_mask(shape + (c["Sq"], c["Skv"]), seed=seed)
        mask[..., c["Sq"] // 2, :] = 1  # a row that sees nothing
    pb = problem_of(c, mask, lens.get("prefix"), lens.get("cu_q"), lens.get("cu_kv"))
    bias = {}
    if alibi:
        bias = dict(alibi=alibi, slopes=np.array(alibi_slopes(c["N"]), dtype=np.float64))
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    o, lse = ref.forward(pb, q, k, v, **bias)
    g = torch.Generator().manual_seed(seed + 1)
    do = torch.randn(o.shape, generator=g).to(torch.bfloat16)
    dlse = torch.randn(lse.shape, generator=g) if with_dlse else None
    t = dict(q=inp["q"], k=inp["k"], v=inp["v"], o=torch.from_numpy(o).to(torch.bfloat16),
             lse=torch.from_numpy(lse).float(), do=do, dlse=dlse, mask=mask)
    want = ref.backward(pb, q, k, v, ref.f64(t["o"]), ref.f64(t["lse"]), ref.f64(do),
                        None if dlse is None else ref.f64(dlse), **bias)
    return c, lens, t, want, bias


def args_of(lens):
    return dict(prefix=lens.get("prefix"), actual_seq_qlen=lens.get("cu_q"),
                actual_seq_kvlen=lens.get("cu_kv"))


def run(c, lens, t, alibi=None, slopes=None, attn=None, **extra):
    d = {k: (None if x is None else x.cuda()) for k, x in t.items()}
    own = attn is None
    attn = attn or fa.MaskedAttention(**c, alibi=alibi)
    try:
        if slopes is not None:
            slopes = torch.tensor(slopes, dtype=torch.float32, device="cuda")
        got = attn.backward(d["do"], d["q"], d["k"], d["v"], d["o"], d["lse"],
                            atten_mask=d["mask"], d_lse=d["dlse"], slopes=slopes, **args_of(lens),
                            **extra)
        torch.cuda.synchronize()
        attn.sync_status()
    finally:
        if own:
            attn.close()
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", sorted(CASES))
def test_backward_matches_formula(name, D):
    c, lens, t, want, _ = setup(name, D, 4000)
    ref.check(run(c, lens, t), want, name)


@pytest.mark.parametrize("name", ["rightdown_dead_rows", "packed", "mask_b1ss"])
def test_gradient_of_lse(name):
    c, lens, t, want, _ = setup(name, 128, 4100, with_dlse=True)
    ref.check(run(c, lens, t), want, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["right", "sqrt", "left"])
@pytest.mark.parametrize("name", ["causal", "rightdown", "band", "prefix", "all", "packed",
                                  "packed_split7", "packed_split8"])
def test_alibi(name, kind, D):
    c, lens, t, want, bias = setup(name, D, 4200, alibi=kind)
    ref.check(run(c, lens, t, alibi=kind, slopes=bias["slopes"]), want, f"{name} {kind}")


@pytest.mark.parametrize("name", ["causal_tiles", "packed", "mask_ss"])
def test_forward_then_backward(name):
    """The chain a training step runs: the kernels' own o and lse go into the
    backward; the wanted gradients are those of the true forward. o and lse
    may each be off by the forward's tolerance: o by 2e-2 at most, which moves
    delta by at most 2e-2 sum |dO|, and lse by 1e-3, a factor on P."""
    c, lens, t, _, _ = setup(name, 128, 4300)
    attn = fa.MaskedAttention(**c)
    d = {k: (None if x is None else x.cuda()) for k, x in t.items()}
    o, lse = attn(d["q"], d["k"], d["v"], atten_mask=d["mask"], **args_of(lens))
    t2 = dict(t, o=o.cpu(), lse=lse.cpu())
    pb = problem_of(c, t["mask"], lens.get("prefix"), lens.get("cu_q"), lens.get("cu_kv"))
    want = ref.backward(pb, *(ref.f64(t[x]) for x in "qkv"), ref.f64(t2["o"]), ref.f64(t2["lse"]),
                        ref.f64(t["do"]))
    ref.check(run(c, lens, t2, attn=attn), want, name)
    attn.close()


def test_alternating_calls_keep_their_lists():
    """One handle, forward and backward in turn with two sets of lengths."""
    N, D = 2, 64
    attn = fa.MaskedAttention("TND", 2, N, 300, 300, D, 3)
    for seed, lens in ((1, [100, 200]), (2, [250, 50]), (1, [100, 200])):
        cu = np.cumsum(lens).tolist()
        c = dict(layout="TND", B=2, N=N, Sq=300, Skv=300, D=D, sparse_mode=3)
        inp = random_inputs("TND", 2, N, 300, 300, D, seed=seed)
        g = torch.Generator().manual_seed(seed)
        do = torch.randn(300, N, D, generator=g).to(torch.bfloat16)
        q, k, v = (inp[x].cuda() for x in "qkv")
        o, lse = attn(q, k, v, actual_seq_qlen=cu, actual_seq_kvlen=cu)
        got = attn.backward(do.cuda(), q, k, v, o, lse, actual_seq_qlen=cu, actual_seq_kvlen=cu)
        pb = problem_of(c, None, None, cu, cu)
        ref.check(got, ref.backward(pb, *(ref.f64(inp[x]) for x in "qkv"), ref.f64(o), ref.f64(lse),
                                    ref.f64(do)), str(lens))
    attn.sync_status()
    attn.close()


@pytest.mark.parametrize("name", ["causal_tiles", "packed", "mask_bnss"])
def test_equal_bits_on_repeat_and_another_stream(name):
    c, lens, t, _, _ = setup(name, 128, 4400)
    a = run(c, lens, t)
    side = torch.cuda.Stream()
    b = run(c, lens, t, stream=side)
    outs = {n: torch.full_like(x, 7.0) for n, x in zip(("dq", "dk", "dv"), a)}
    e = run(c, lens, t, stream=side.cuda_stream, **outs)
    for x, y, z in zip(a, b, e):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_many_items_claimed_order():
    """1,300 packed sequences x 2 heads: lists of several items per SM."""
    g = torch.Generator().manual_seed(4500)
    lens = torch.randint(1, 260, (1300,), generator=g)
    cu = torch.cumsum(lens, 0).tolist()
    c = dict(layout="TND", B=1300, N=2, Sq=cu[-1], Skv=cu[-1], D=64, sparse_mode=3)
    inp = random_inputs("TND", 1300, 2, cu[-1], cu[-1], 64, seed=4501)
    do = torch.randn(cu[-1], 2, 64, generator=g).to(torch.bfloat16)
    q, k, v = (inp[x].cuda() for x in "qkv")
    attn = fa.MaskedAttention(**c)
    o, lse = attn(q, k, v, actual_seq_qlen=cu, actual_seq_kvlen=cu)
    got = attn.backward(do.cuda(), q, k, v, o, lse, actual_seq_qlen=cu, actual_seq_kvlen=cu)
    attn.sync_status()
    pb = problem_of(c, None, None, cu, cu)
    ref.check(got, ref.backward(pb, *(ref.f64(inp[x]) for x in "qkv"), ref.f64(o), ref.f64(lse),
                                ref.f64(do)))
    attn.close()


def test_nan_of_another_sequence_stays_there():
    """Sequences share tiles of packed tokens: what the neighbour's rows hold
    does not reach this sequence's gradients."""
    c = dict(layout="TND", B=3, N=2, Sq=300, Skv=330, D=128, sparse_mode=3)
    cu_q, cu_kv = [70, 170, 300], [80, 190, 330]
    inp = random_inputs("TND", 3, 2, 300, 330, 128, seed=4600)
    g = torch.Generator().manual_seed(4601)
    do = torch.randn(300, 2, 128, generator=g).to(torch.bfloat16)
    pb = problem_of(c, None, None, cu_q, cu_kv)
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    o, lse = ref.forward(pb, q, k, v)
    o, lse = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()
    want = ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do))
    t = {"q": inp["q"], "k": inp["k"], "v": inp["v"], "o": o, "do": do}
    t = {n: x.clone() for n, x in t.items()}
    for n in ("q", "o", "do"):
        t[n][70:170] = float("nan")
    for n in ("k", "v"):
        t[n][80:190] = float("inf")
    got = run(c, dict(cu_q=cu_q, cu_kv=cu_kv), dict(t, lse=lse, dlse=None, mask=None))
    for name, x, (a, z) in zip(("dq", "dk", "dv"), got, ((70, 170), (80, 190), (80, 190))):
        x = x.clone()
        x[a:z] = 0
        value, bound = (y.copy() for y in want[name])
        value[a:z] = bound[a:z] = 0
        ref.check([x], {name: (value, bound)}, "neighbours")


def test_refusals_touch_nothing():
    c, lens, t, _, _ = setup("causal", 64, 4700)
    d = {k: (None if x is None else x.cuda()) for k, x in t.items()}
    attn = fa.MaskedAttention(**c)
    dq = torch.full_like(d["q"], 3.0)
    base = (d["do"], d["q"], d["k"], d["v"], d["o"], d["lse"])
    for i in range(6):
        for bad in (base[i].cpu(), base[i].double(), base[i][..., :-1].contiguous(),
                    base[i].transpose(0, 1)):
            with pytest.raises(ValueError):
                attn.backward(*base[:i], bad, *base[i + 1:], dq=dq)
    with pytest.raises(ValueError):
        attn.backward(*base, dq=dq, d_lse=d["lse"].double())
    with pytest.raises(fa.FaError) as e:  # slopes on a handle without ALiBi
        attn.backward(*base, dq=dq, slopes=torch.ones(c["N"], device="cuda"))
    assert e.value.name == "FA_ERR_PARAM_INVALID"
    with pytest.raises(fa.FaError) as e:  # a graph would replay another call's work list
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            attn.backward(*base, dq=dq)
    assert e.value.name == "FA_ERR_UNSUPPORTED"
    torch.cuda.synchronize()
    assert (dq == 3.0).all()
    attn.close()
    al = fa.MaskedAttention(**c, alibi="right")
    with pytest.raises(fa.FaError) as e:
        al.backward(*base, dq=dq)
    assert e.value.name == "FA_ERR_PARAM_INVALID"
    al.close()


def test_no_tokens_on_a_side():
    """No query rows: dk and dv are zero. No keys: dq is zero."""
    z = dict(dtype=torch.bfloat16, device="cuda")
    attn = fa.MaskedAttention("BNSD", 1, 2, 0, 130, 64, 0)
    k = torch.randn(1, 2, 130, 64, **z)
    e = torch.empty(1, 2, 0, 64, **z)
    dq, dk, dv = attn.backward(e, e, k, k, e, torch.empty(1, 2, 0, device="cuda"),
                               dk=torch.ones_like(k), dv=torch.ones_like(k))
    assert dq.numel() == 0 and not dk.any() and not dv.any()
    attn.sync_status()
    attn.close()
    attn = fa.MaskedAttention("BNSD", 1, 2, 130, 0, 64, 0)
    lse = torch.full((1, 2, 130), -float("inf"), device="cuda")
    dq, dk, dv = attn.backward(k, k, e, e, k, lse, dq=torch.ones_like(k))
    assert not dq.any() and dk.numel() == 0
    attn.sync_status()
    attn.close()
