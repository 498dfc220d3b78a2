"""Attention over the quantised cache where sizes are far apart, against the
64-bit form, in test_attend_gpu's way."""
import pytest

from test_attend_gpu import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 128)])
@pytest.mark.parametrize("hidden", [200.0, 60000.0])
def test_a_hidden_key_takes_no_bits(heads, dim, hidden):
    """Keys of 10^-4 under queries of 10^4; the next drafted token's key, which
    the token before it does not see, is far above them."""
    B = 5
    with Step([2, 3, 2, 2, 4], [9, 40, 70, 130, 20], [-1, 0, -1, 0, 0], [33], heads, 2, dim, 16, "f16", kscale=1e-4,
              qscale=6e3, spread=0.3) as s:
        for b in range(B):
            at = s.kv_len[b] - 1
            s.k_in[s.pages[b][at // 16] * 16 + at % 16] = hidden
        s.write()
        out, lse = s.run()
        last = {sum(s.q_len[:b + 1]) - 1 for b in range(B)}  # these see it
        s.check(out, lse, tokens=set(range(s.T)) - last)
