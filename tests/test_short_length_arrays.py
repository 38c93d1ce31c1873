"""Length and prefix arrays with fewer entries than the problem has batch entries:
refused by the binding, whose C library would read past their end. Arrays that the
problem does not take, and longer ones, are accepted as before. No GPU: the check
comes before the tensors are looked at."""
import numpy as np
import pytest
import torch

import masked_attention_fa_b200 as fa

PACKED = dict(layout="TND", B=3, N=2, Sq=30, Skv=30, D=64, sparse_mode=3)
PREFIX = dict(layout="BNSD", B=3, N=2, Sq=30, Skv=30, D=64, sparse_mode=5)
FULL = dict(actual_seq_qlen=[10, 20, 30], actual_seq_kvlen=[10, 20, 30])
SHORT = [dict(FULL, actual_seq_qlen=[10, 30]), dict(FULL, actual_seq_kvlen=np.array([30])),
         dict(FULL, actual_seq_qlen=torch.tensor([10, 30]))]


def calls(c):
    x = torch.zeros(1, dtype=torch.bfloat16)
    attn = fa.MaskedAttention(**c)
    yield "forward", lambda **kw: attn(x, x, x, **kw)
    yield "bias", lambda **kw: attn(x, x, x, rel_bias=x, rel_buckets=[0, 0, 0], **kw)
    yield "backward", lambda **kw: attn.backward(x, x, x, x, x, x, **kw)
    if c["layout"] == "TND":
        yield "paged", lambda **kw: attn.paged(x, x, x, x, kw.pop("actual_seq_qlen"),
                                               kw.pop("actual_seq_kvlen"), **kw)
    desc = fa.make_desc(**c)
    for f in (fa.fa_validate, fa.fa_visible_pairs, fa.fa_plan_stats, fa.fa_plan_items):
        yield f.__name__, lambda f=f, **kw: f(desc, **kw)


@pytest.mark.parametrize("kw", SHORT, ids=["list", "array", "torch"])
def test_packed(kw):
    for name, call in calls(PACKED):
        with pytest.raises(ValueError, match="entries"):
            call(**kw)


def test_prefix():
    for name, call in calls(PREFIX):
        with pytest.raises(ValueError, match="prefix has 2 entries"):
            call(prefix=[1, 2])


def test_others_are_accepted():
    longer = {k: v + [30] for k, v in FULL.items()}
    desc = fa.make_desc(**PACKED)
    assert fa.fa_validate(desc, **longer) == 0
    assert fa.fa_visible_pairs(desc, **longer) == fa.fa_visible_pairs(desc, **FULL)
    assert fa.fa_validate(desc, prefix=[1], **FULL) == 0
    assert fa.fa_validate(fa.make_desc(**dict(PREFIX, sparse_mode=2)), prefix=[1],
                          actual_seq_qlen=[3]) == 0
    one = fa.make_desc(**dict(PREFIX, B=1))
    assert fa.fa_validate(one, prefix=7) == 0  # a number stands for an array of one
    assert fa.fa_validate(one, prefix=torch.tensor([7])) == 0
    assert fa.fa_validate(one, prefix=np.array([[7]])) == 0
