"""A batch that the binding refuses leaves the plan as it was: outputs that are
too short for the batch before are refused, and right ones get its results."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_tree_gpu import TreeStep

pytestmark = pytest.mark.gpu


def test_refused_batches_leave_the_plan_before():
    with TreeStep(["near", "star"], [6, 3], [40, 11], [-1, -1], [], 4, 2, 64, 16, "f16") as s:
        want, want_lse = s.run()
        parent, lists = s.parent(), s.lists()
        for bad in (None, parent[:-1], parent.long(), parent.repeat(2)[::2], parent.cuda()):
            with pytest.raises(ValueError, match="parent"):
                lora.lora_attend_plan_set_tree(s.plan, s.kv, bad, **lists)
            for short in (want[:0], want[:8]):
                with pytest.raises(ValueError, match="out"):
                    lora.lora_attend(s.kv, s.plan, s.q, s.scale, short.clone())
            with pytest.raises(ValueError, match="q:"):
                lora.lora_attend(s.kv, s.plan, s.q[:8], s.scale, torch.empty_like(want))
            with pytest.raises(ValueError, match="lse"):
                lora.lora_attend(s.kv, s.plan, s.q, s.scale, torch.empty_like(want), want_lse[:8].clone())
            out, lse = torch.empty_like(want), torch.empty_like(want_lse)
            lora.lora_attend(s.kv, s.plan, s.q, s.scale, out, lse)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
