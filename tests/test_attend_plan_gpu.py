"""What a plan is after a refusal, and what captured calls make of later plans."""
import ctypes

import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_attend_gpu import Step

pytestmark = pytest.mark.gpu


def test_every_refusal_leaves_no_plan():
    """A cache of other heads, no cache, no batch, a bad list, a capture: the
    batch before is not attended to again."""
    lib, f = lora.raw_lib(), ctypes.c_float
    with Step([1, 1], [20, 40], [-1, 0], [33], 4, 2, 64, 16, "f16") as s:
        out = torch.full((2, 4, 64), 7.0, dtype=torch.float16, device="cuda")

        def attend():
            return lib.lora_attend(s.kv, s.plan, s.q.data_ptr(), 320, f(1), out.data_ptr(), None, None)
        wide = lora.lora_kv_create(s.n_pages, 16, 2, 128, torch.float16)
        more = lora.lora_kv_create(s.n_pages, 16, 4, 64, torch.float16)
        b = lora.lora_attend_batch()
        st = torch.cuda.Stream()

        def captured():
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
                x = out * 2  # a graph of one node
                s.set_plan()
            return x
        refusals = [(lora.LORA_EMISMATCH, lambda: lora.lora_attend_plan_set(s.plan, wide, **s.lists())),
                    (lora.LORA_EMISMATCH, lambda: lora.lora_attend_plan_set(s.plan, more, **s.lists())),
                    (lora.LORA_EINVAL, lambda: lora.lora_attend_plan_set(s.plan, None, **s.lists())),
                    (lora.LORA_EINVAL, lambda: lora.lora_attend_plan_set(
                        s.plan, s.kv, **dict(s.lists(), kv_len=torch.tensor([20, -1], dtype=torch.int32)))),
                    (lora.LORA_EINVAL, captured)]
        try:
            for status, refused in refusals:
                s.set_plan()
                with pytest.raises(lora.LoraError) as e:
                    refused()
                assert e.value.status == status
                assert attend() == lora.LORA_EINVAL
            s.set_plan()
            assert lib.lora_attend_plan_set(s.plan, s.kv, None, None) == lora.LORA_EINVAL
            assert attend() == lora.LORA_EINVAL
            assert lib.lora_attend_plan_set(None, s.kv, ctypes.byref(b), None) == lora.LORA_EINVAL
            torch.cuda.synchronize()
            assert (out == 7).all()
            s.check(*s.run())
        finally:
            lora.lora_kv_destroy(wide)
            lora.lora_kv_destroy(more)
