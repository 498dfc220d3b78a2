"""Tables whose farthest angles overflow: refused, since they have no cosine."""
import pytest

from rank_adapter_gemm_token_amd import lora
from test_append_cpu import create


@pytest.mark.parametrize("n,freq", [(3, 1.7e308), (1 << 24, 2e301), (1 << 24, -2e301)])
def test_angles_that_overflow(n, freq):
    assert create(n=n, rot=16, freq=(1.0,) * 7 + (freq,)) == lora.LORA_EINVAL
