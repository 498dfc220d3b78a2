"""The binding's checks of the attention plan's and the verification's
arguments, made before the library is called."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.fixture
def no_plan():
    """A plan of the binding's that the library knows as NULL, which it refuses."""
    lora._attend_plans[None] = [4, 64, 0]
    yield None
    del lora._attend_plans[None]


def test_page_lists_are_as_long_as_the_batch_s_last_bound(no_plan):
    """page0 may be longer than the batch needs (a buffer kept for the largest
    one): the entry after the last sequence's counts, not the buffer's last."""
    one, none = i32(1, 1), i32(-1, -1)

    def plan_set(pages, page0, **prefix):
        lora.lora_attend_plan_set(no_plan, None, one, i32(20, 20), none, pages, page0, stream=0, **prefix)
    with pytest.raises(ValueError, match="pages: expected 4"):
        plan_set(i32(3), i32(0, 2, 4, 0, 0))
    with pytest.raises(lora.LoraError):  # long enough for its two sequences: the library's turn
        plan_set(i32(3, 2, 1, 0), i32(0, 2, 4, 99))
    good = dict(pages=i32(3, 2, 1, 0), page0=i32(0, 2, 4), prefix_len=i32(30))
    with pytest.raises(ValueError, match="prefix_pages: expected 2"):
        plan_set(**good, prefix_pages=i32(5), prefix_page0=i32(0, 2, 0))
    with pytest.raises(lora.LoraError):
        plan_set(**good, prefix_pages=i32(5, 6), prefix_page0=i32(0, 2, 99))


def test_bounds_are_looked_at_after_their_type_is(no_plan):
    one = i32(1, 1)
    for page0 in (i32(0, 2, 4).long(), i32(0, 2), None, i32(0, 0, 2, 0, 4)[::2]):
        with pytest.raises(ValueError, match="page0"):
            lora.lora_attend_plan_set(no_plan, None, one, one, one, i32(1, 2, 3, 4), page0)
        with pytest.raises(ValueError, match="prefix_page0"):
            lora.lora_attend_plan_set(no_plan, None, one, one, one, i32(1, 2, 3, 4), i32(0, 2, 4), one,
                                      i32(1, 2, 3, 4), page0)


def test_the_draft_has_the_target_s_vocabulary():
    """Rows of another length would be read at the wrong stride.  Without
    drafted tokens the draft is not looked at."""
    p, i = torch.zeros(4, 64), i32(0, 0, 0, 0)
    for wrong in (torch.zeros(2, 96), torch.zeros(4, 32), torch.zeros(128)):
        with pytest.raises(ValueError, match="p_draft: .* vocabulary"):
            lora.lora_verify(None, p, wrong, i, i, p, 2, 4, i, i, stream=0)
    for q in (torch.zeros(2, 64), torch.zeros(1, 2, 64)):
        with pytest.raises(ValueError, match="p_target: .* on the device"):
            lora.lora_verify(None, p, q, i, i, p, 2, 4, i, i, stream=0)
    with pytest.raises(ValueError, match="p_target: .* on the device"):
        lora.lora_verify(None, p, torch.zeros(0, 7), i, i, p, 4, 4, i, i, stream=0)
