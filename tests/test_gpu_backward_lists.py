"""The backward pass's work lists: items without a tile between items with
some (planes of a mask that hide everything), many items per SM, short and long
ones mixed. The items are claimed at run time, so every case runs often: equal
bits each time, and no device-side wait gives up."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from gpu_helpers import problem_of
from masked_attention_fa_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def masked(pattern, B, N, sq, skv, seed):
    """uint8 [B, N, sq, skv] masks: planes that hide everything, but for some
    of them, or some key or query tiles of every plane."""
    g = torch.Generator().manual_seed(seed)
    m = torch.ones(B, N, sq, skv, dtype=torch.uint8)
    if pattern == "planes":
        for x in range(0, B * N, 9):
            m[x // N, x % N] = (torch.rand(sq, skv, generator=g) < 0.3).to(torch.uint8)
    elif pattern == "keys":
        m[..., skv - 130:skv - 100] = 0
    elif pattern == "rows":
        m[:, :, 131:133] = (torch.rand(B, N, 2, skv, generator=g) < 0.5).to(torch.uint8)
    return m


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pattern", ["planes", "keys", "rows", "nothing"])
def test_items_without_tiles_between_others(pattern, D):
    B, N, sq, skv = 2, 41, 515, 640
    c = dict(layout="BNSD", B=B, N=N, Sq=sq, Skv=skv, D=D, sparse_mode=1, mask_kind="BNSS")
    inp = random_inputs("BNSD", B, N, sq, skv, D, seed=8000)
    mask = masked(pattern, B, N, sq, skv, 8001)
    pb = problem_of(c, mask)
    q, k, v = (ref.f64(inp[x]) for x in "qkv")
    o, lse = ref.forward(pb, q, k, v)
    o, lse = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(8002)).to(torch.bfloat16)
    want = ref.backward(pb, q, k, v, ref.f64(o), ref.f64(lse), ref.f64(do))
    a = [x.cuda() for x in (do, inp["q"], inp["k"], inp["v"], o, lse)]
    gm = mask.cuda()
    attn = fa.MaskedAttention(**c)
    first = attn.backward(*a, atten_mask=gm)
    ref.check(first, want, pattern)
    for _ in range(40):
        for x, y in zip(first, attn.backward(*a, atten_mask=gm)):
            assert torch.equal(x, y)
    attn.sync_status()
    attn.close()


@pytest.mark.parametrize("D", [64, 128])
def test_long_and_short_items_often(D):
    """Sequences of 1 to 1,500 tokens, calls queued behind each other."""
    g = np.random.default_rng(8100)
    lens = np.concatenate([g.integers(1, 140, 60), g.integers(900, 1500, 6), np.zeros(9, np.int64)])
    g.shuffle(lens)
    cu = np.cumsum(lens).tolist()
    c = dict(layout="TND", B=len(lens), N=4, Sq=cu[-1], Skv=cu[-1], D=D, sparse_mode=3)
    inp = random_inputs("TND", c["B"], 4, cu[-1], cu[-1], D, seed=8101)
    attn = fa.MaskedAttention(**c)
    q, k, v = (inp[x].cuda() for x in "qkv")
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(8102)).to(torch.bfloat16).cuda()
    lens = dict(actual_seq_qlen=cu, actual_seq_kvlen=cu)
    o, lse = attn(q, k, v, **lens)
    first = attn.backward(do, q, k, v, o, lse, **lens)
    pb = problem_of(c, None, None, cu, cu)
    ref.check(first, ref.backward(pb, *(ref.f64(inp[x]) for x in "qkv"), ref.f64(o), ref.f64(lse),
                                  ref.f64(do)))
    results = [attn.backward(do, q, k, v, o, lse, **lens) for _ in range(60)]
    attn.sync_status()
    for r in results:
        for x, y in zip(first, r):
            assert torch.equal(x, y)
    attn.close()
