"""Backward calls that are allowed though unusual: operands and gradients that
are views 16 bytes into a buffer, a mask at an odd byte, a call after one that
failed half-way on another stream; and the refusal of overlapping outputs."""
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


def shifted(t, by):
    """t's values `by` elements into a buffer filled with another value."""
    buf = torch.full((t.numel() + 2 * by,), 7, dtype=t.dtype, device=t.device)
    out = buf[by:by + t.numel()].view(t.shape)
    out.copy_(t)
    return out, buf


def operands(c, seed, cu_q=None, cu_kv=None, table=None, buckets=None, mask=None):
    inp = random_inputs(c["layout"], c["B"], c["N"], c["Sq"], c["Skv"], c["D"], seed=seed)
    kw = dict(table=ref.f64(table), bucket_of=buckets) if table is not None else {}
    o, lse = ref.forward(problem_of(c, mask, None, cu_q, cu_kv),
                         *(ref.f64(inp[x]) for x in "qkv"), **kw)
    o, lse = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()
    g = torch.Generator().manual_seed(seed + 1)
    do = torch.randn(o.shape, generator=g).to(torch.bfloat16)
    return [x.cuda() for x in (do, inp["q"], inp["k"], inp["v"], o, lse)]


# The last writes dS out (more than four items per SM).
@pytest.mark.parametrize("N,S,D", [(2, 301, 64), (2, 301, 128), (60, 700, 128)])
def test_views_sixteen_bytes_into_a_buffer(N, S, D):
    c = dict(layout="BSND", sparse_mode=3, B=1, N=N, Sq=S, Skv=S + 30, D=D)
    t = operands(c, 7100)
    attn = fa.MaskedAttention(**c)
    want = attn.backward(*t)
    views = [shifted(x, 8 if x.dtype is torch.bfloat16 else 1)[0] for x in t]
    outs = [shifted(torch.zeros_like(x), 8) for x in want]
    got = attn.backward(*views, dq=outs[0][0], dk=outs[1][0], dv=outs[2][0])
    torch.cuda.synchronize()
    attn.sync_status()
    for a, b, (_, buf) in zip(got, want, outs):
        assert torch.equal(a, b)
        assert (buf[:8] == 7).all() and (buf[-8:] == 7).all()
    o = shifted(t[4], 8)[0]
    plain, moved = attn(*t[1:4]), attn(*views[1:4], out=o)
    assert torch.equal(plain[0], moved[0]) and torch.equal(plain[1], moved[1])
    attn.close()


@pytest.mark.parametrize("by", [1, 2, 3])
def test_mask_at_an_odd_byte(by):
    c = dict(layout="BNSD", sparse_mode=1, B=2, N=2, Sq=200, Skv=333, D=64, mask_kind="B1SS")
    mask = (torch.rand(2, 1, 200, 333, generator=torch.Generator().manual_seed(3)) < 0.4)
    mask = mask.to(torch.uint8)
    t = operands(c, 7200, mask=mask)
    attn = fa.MaskedAttention(**c)
    want = attn.backward(*t, atten_mask=mask.cuda())
    got = attn.backward(*t, atten_mask=shifted(mask.cuda(), by)[0])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    attn.close()


def test_bad_alignment_and_overlaps_are_refused():
    c = dict(layout="BNSD", sparse_mode=2, B=1, N=2, Sq=140, Skv=140, D=64)
    table = torch.randn(8, 2, generator=torch.Generator().manual_seed(1))
    m = fa.relative_buckets(8, 20)
    t = operands(c, 7300, table=table, buckets=m)
    table = table.cuda()
    kept = [x.clone() for x in t]
    attn = fa.MaskedAttention(**c)

    def refused(args, **kw):
        with pytest.raises(fa.FaError) as e:
            attn.backward(*args, rel_bias=table, rel_buckets=m, **kw)
        assert e.value.name == "FA_ERR_PARAM_INVALID"

    for i in range(5):
        for by in (1, 4):  # 2 and 8 bytes
            refused(t[:i] + [shifted(t[i], by)[0]] + t[i + 1:])
    dq, dk = torch.empty_like(t[1]), torch.empty_like(t[2])
    for name in ("dq", "dk", "dv"):
        refused(t, **{name: shifted(t[1], 4)[0]})
        for x in t[:5]:
            refused(t, **{name: x})
    refused(t, dk=dk, dv=dk)
    refused(t, dq=dq, dv=dq)
    refused(t, d_rel_bias=table)
    both = torch.empty(2 * dq.numel(), dtype=dq.dtype, device="cuda")
    part = lambda at: both[at:at + dq.numel()].view(dq.shape)
    refused(t, dk=part(0), dv=part(dq.numel() - 8))
    attn.backward(*t, rel_bias=table, rel_buckets=m, dk=part(0), dv=part(dq.numel()))
    torch.cuda.synchronize()
    attn.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(t, kept))
    attn.close()


def test_call_after_one_that_failed_on_another_stream(monkeypatch):
    """A call uploads its work list on a busy stream and then finds no memory:
    a call elsewhere waits for the list."""
    D, N, S = 64, 2, 500
    c = dict(layout="TND", sparse_mode=3, B=2, N=N, Sq=S, Skv=S, D=D)
    first, then = [130, S], [370, S]  # as many tiles, so that the list's buffer stays
    table = torch.randn(8, N, generator=torch.Generator().manual_seed(2))
    near, far = fa.relative_buckets(8, 20), fa.relative_buckets(8, 900)
    t1 = operands(c, 7400, first, first, table, near)
    t2 = operands(c, 7400, then, then, table, near)
    table = table.cuda()
    fresh = fa.MaskedAttention(**c)
    want = fresh.backward(*t2, rel_bias=table, rel_buckets=near, actual_seq_qlen=then,
                          actual_seq_kvlen=then)
    torch.cuda.synchronize()
    fresh.close()
    attn = fa.MaskedAttention(**c)
    attn.backward(*t1, rel_bias=table, rel_buckets=near, actual_seq_qlen=first,
                  actual_seq_kvlen=first)
    torch.cuda.synchronize()
    busy = torch.cuda.Stream()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(100_000_000)
    monkeypatch.setenv("FA_TEST_FAIL_ALLOC", "1")
    with pytest.raises(fa.FaError) as e:  # a farther reach needs a larger workspace
        attn.backward(*t2, rel_bias=table, rel_buckets=far, actual_seq_qlen=then,
                      actual_seq_kvlen=then, stream=busy)
    assert e.value.name == "FA_ERR_ALLOC"
    monkeypatch.delenv("FA_TEST_FAIL_ALLOC")
    got = attn.backward(*t2, rel_bias=table, rel_buckets=near, actual_seq_qlen=then,
                        actual_seq_kvlen=then)
    torch.cuda.synchronize()
    attn.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    attn.close()
