"""Plans of the token mixers with one status word (plans on the CPU: nothing is launched)."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()


def test_plans_share_a_word():
    a = B.LinearAttention(1, 6, 4, 64, 64, device="cpu")
    b = B.LinearAttention(1, 9, 4, 64, 64, device="cpu", word=a.word)
    c = B.PromptAttention(1, 9, 4, 2, 64, device="cpu", word=a.word)
    d = B.PromptAttention(1, 9, 4, 2, 64, device="cpu")
    assert a.desc.status == b.desc.status == c.desc.status == a.word.data_ptr() != d.desc.status
    # and so have the descriptors that calls with other row distances hand to the library
    assert all(p._ref((1, 2, 3, 4, 5, 6))._obj.status == a.word.data_ptr() for p in (a, b, c))


@pytest.mark.parametrize("bad", [torch.zeros(4), torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)[::2]])
def test_other_words_are_refused(bad):
    with pytest.raises(ValueError, match="word"):
        B.LinearAttention(1, 6, 4, 64, 64, device="cpu", word=bad)
