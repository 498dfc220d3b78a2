"""What the binding knows of an attention plan's batch after a call: the
library's batch, whichever of the two refused the new one."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


LISTS = dict(q_len=i32(2, 2), kv_len=i32(2, 2), group=i32(-1, -1), pages=i32(0, 1), page0=i32(0, 1, 2))
BAD_PARENTS = [None, i32(-1, 0, -1), i32(-1, 0, -1, 0).long(), i32(-1, 9, 0, 9, -1, 9, 0, 9)[::2], torch.zeros(4)]


@pytest.fixture
def plan():
    """A plan of the binding's, of six tokens, that the library knows as NULL."""
    lora._attend_plans[None] = [4, 64, 6]
    yield None
    del lora._attend_plans[None]


@pytest.mark.parametrize("bad", BAD_PARENTS, ids=["none", "short", "int64", "strided", "float"])
def test_refused_parents_leave_the_batch_before(plan, bad):
    with pytest.raises(ValueError, match="parent"):
        lora.lora_attend_plan_set_tree(plan, None, bad, **LISTS, stream=0)
    assert lora._attend_plans[plan] == [4, 64, 6]


@pytest.mark.parametrize("change", [dict(kv_len=i32(2)), dict(group=i32(-1, -1).long()), dict(pages=i32(0)),
                                    dict(page0=i32(0, 1)), dict(prefix_len=i32(3)), dict(stream="none")],
                         ids=["kv_len", "group", "pages", "page0", "prefix", "stream"])
@pytest.mark.parametrize("tree", [False, True])
def test_refused_lists_leave_the_batch_before(plan, change, tree):
    lists = {**LISTS, "stream": 0, **change}
    with pytest.raises((ValueError, AttributeError)):
        if tree:
            lora.lora_attend_plan_set_tree(plan, None, i32(-1, 0, -1, 0), **lists)
        else:
            lora.lora_attend_plan_set(plan, None, **lists)
    assert lora._attend_plans[plan] == [4, 64, 6]


@pytest.mark.parametrize("tree", [False, True])
def test_arguments_that_reach_no_library_leave_the_batch_before(plan, tree):
    """No handle: the call cannot be made."""
    with pytest.raises(Exception) as e:
        if tree:
            lora.lora_attend_plan_set_tree(plan, 1.5, i32(-1, 0, -1, 0), **LISTS, stream=0)
        else:
            lora.lora_attend_plan_set(plan, 1.5, **LISTS, stream=0)
    assert not isinstance(e.value, lora.LoraError)
    assert lora._attend_plans[plan] == [4, 64, 6]


@pytest.mark.parametrize("tree", [False, True])
def test_the_library_s_refusal_leaves_no_tokens(plan, tree):
    with pytest.raises(lora.LoraError):
        if tree:
            lora.lora_attend_plan_set_tree(plan, None, i32(-1, 0, -1, 0), **LISTS, stream=0)
        else:
            lora.lora_attend_plan_set(plan, None, **LISTS, stream=0)
    assert lora._attend_plans[plan] == [4, 64, 0]
