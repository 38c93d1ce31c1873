"""Room for dS (head dim 128, more than 4 work items per SM): with less memory
than the whole, smaller shares and the same bits; with less than one head's, two
walks, whose dq is another order of the same sums; and neither for longer than
the lengths that met it: a handle that had no room once writes dS again."""
import pytest
import torch

import masked_attention_fa_b200 as fa
import training_reference as ref
from test_gpu_backward_spill import run, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from masked_attention_fa_b200 import build
    build.build()
    fa.load_library()


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name,bias", [("packed", None), ("mask_bnss", None), ("prefix", "learned"),
                                       ("causal", "right")])
def test_less_room(name, bias, monkeypatch):
    c, lens, mask, t, want, call = setup(name, bias)
    whole = run(c, lens, mask, t, call)
    for tiles in (100, 37, 24):  # of 128 x 128; a head takes at most 12
        monkeypatch.setenv("FA_TEST_SPILL_ROOM", str(tiles))
        assert equal(whole, run(c, lens, mask, t, call))
    monkeypatch.setenv("FA_TEST_SPILL_ROOM", "0")
    walks = run(c, lens, mask, t, call)
    assert equal(whole[1:], walks[1:])
    ref.check(walks, want, name)


def test_no_room_does_not_last(monkeypatch):
    c, lens, mask, t, want, call = setup("packed")
    whole = run(c, lens, mask, t, call)
    monkeypatch.setenv("FA_TEST_SPILL_ROOM", "0")
    attn = fa.MaskedAttention(**c)
    walks = run(c, lens, mask, t, call, attn)
    assert not torch.equal(walks[0], whole[0])  # or the test tells nothing apart
    monkeypatch.delenv("FA_TEST_SPILL_ROOM")
    assert equal(run(c, lens, mask, t, call, attn), walks)  # a repeated call keeps its bits
    one = dict(cu_q=[c["Sq"]] * c["B"], cu_kv=[c["Skv"]] * c["B"])
    run(c, one, mask, t, call, attn)
    assert equal(run(c, lens, mask, t, call, attn), whole)
    attn.close()
