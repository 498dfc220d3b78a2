"""Attention over the quantised cache where sizes are far apart, against the
64-bit form, in test_attend_gpu's way."""
import numpy as np
import pytest
import torch

from rank_adapter_gemm_token_amd import lora
from test_attend_gpu import DT, Step

pytestmark = pytest.mark.gpu


def light_and_heavy(dtype, per):
    """Output and lse of 300 sequences over the same 2^19 keys: one of score 18,
    the others 0; all values 1.  So many sequences, on the same pages, that each
    is one wave's work."""
    n, page, dim, kv_heads, B = 1 << 19, 1024, 64, 8, 300
    heads, pages = kv_heads * per, n // page
    kv = lora.lora_kv_create(pages, page, kv_heads, dim, dtype)
    plan = lora.lora_attend_plan_create(B, 0, B, B * pages, heads, kv_heads, dim)
    try:
        k, v = (torch.full((n, kv_heads, dim), x, dtype=dtype, device="cuda") for x in (0.0, 1.0))
        k[0, :, 3] = 18.0
        lora.lora_kv_write(kv, k, v, torch.arange(n, dtype=torch.int32, device="cuda"), n)

        def i32(x):
            return torch.tensor(x, dtype=torch.int32)
        lora.lora_attend_plan_set(plan, kv, i32([1] * B), i32([n] * B), i32([-1] * B),
                                  torch.arange(pages, dtype=torch.int32).repeat(B),
                                  torch.arange(B + 1, dtype=torch.int32) * pages)
        q = torch.zeros((B, heads, dim), dtype=dtype, device="cuda")
        q[:, :, 3] = 1.0
        out, lse = torch.empty_like(q), torch.empty((B, heads), device="cuda")
        lora.lora_attend(kv, plan, q, 1.0, out, lse)
        return out.double().cpu().numpy(), lse.double().cpu().numpy()
    finally:
        torch.cuda.synchronize()
        lora.lora_attend_plan_destroy(plan)
        lora.lora_kv_destroy(kv)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("per", [1, 32])
def test_many_light_keys_stay_in_the_sum(dtype, per):
    """2^19 weights of e^-18 beside one of 1 are 1/128 of the sum, though each
    alone is below fp32's half step at 1: one rounding of 2^-24 a tile of 64
    keys (2^13 of them), beside that of the logarithm's terms."""
    _, lse = light_and_heavy(DT[dtype], per)
    want = 18.0 + np.log1p(((1 << 19) - 1) * np.exp(-18.0))
    assert np.abs(lse - want).max() <= 2.0 ** -11 + 2.0 ** -14


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("per", [1, 32])
def test_many_light_keys_stay_in_the_output(dtype, per):
    """Light keys hold 1/128 of the whole, and all values are 1: the output is
    1, to its own rounding and that of the weights (half a step of fp16, 2^-11;
    with 32 rows the largest weight may stand at 2^7, so a light one is off by
    up to 2^-25 of 2^7: 2^17 2^-32 for a quarter of them; 2^-16 for the rest)."""
    out, _ = light_and_heavy(DT[dtype], per)
    tol = torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -16
    assert np.abs(out - 1).max() <= tol, np.abs(out - 1).max()


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


WIDE = [2.0 ** 60, 2.0 ** 71, 2.0 ** 80, 2.0 ** 100, 2.0 ** 120]


@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (8, 1, 128), (64, 2, 64)])
@pytest.mark.parametrize("vscale", WIDE)
@pytest.mark.parametrize("kscale", [0.0, 1.0])
def test_rows_of_zeros_beside_huge_ones(heads, kv_heads, dim, vscale, kscale):
    """Their weights stay in the sum: in a tile, in another wave's tiles, in the
    prefix beside huge own values and the other way round, before and after."""
    with Step([1, 2, 1, 1, 1], [333, 40, 700, 90, 130], [0, 0, -1, 1, 1], [260, 70], heads, kv_heads, dim, 16, "bf16",
              kscale=kscale, vscale=vscale / 16, spread=0.5) as s:
        def slots(pages):
            return [p * 16 + i for p in pages for i in range(16)]
        s.v_in[slots(s.prefix_pages[0])] = 0       # a prefix of zeros before huge values
        for at in (slots(s.pages[3]), slots(s.pages[4])):
            s.v_in[at] = 0                         # zeros after a huge prefix
        mixed = slots(s.pages[2])
        s.v_in[mixed[::3]] = 0
        s.v_in[mixed[:300]] = 0                    # some tiles of nothing else, first
        s.v_in[slots(s.pages[1])[1::2]] = 0
        s.write()
        s.check(*s.run())


@pytest.mark.parametrize("low,high", [(-64, 64), (-40, 100), (-70, 118)])
def test_value_exponents_of_the_whole_range(low, high):
    """Value rows of exponents from the least to the largest, in any order."""
    with Step([1, 3, 1], [500, 90, 1111], [0, 0, -1], [300], 4, 2, 64, 16, "bf16", spread=0.3) as s:
        e = torch.randint(low, high + 1, (s.v_in.shape[0], s.kv_heads, 1), generator=torch.Generator().manual_seed(3))
        s.v_in = torch.ldexp(s.v_in.float(), e).to(s.dtype)
        s.write()
        s.check(*s.run())


def test_light_huge_values_beside_heavy_small_ones():
    """Values of 2^90 whose weight is 2^-100 to 2^-200 of the others', of 2^-20:
    they decide the outputs or do not count, as the products say."""
    for gap in (60.0, 80.0, 100.0, 140.0):
        with Step([1, 2], [200, 70], [0, -1], [100], 4, 2, 64, 16, "bf16", kscale=0.05, vscale=2.0 ** -20,
                  spread=0.3) as s:
            q = torch.zeros_like(s.q)
            q.copy_(s.q * 0.01)
            q[..., 0] = 1.0
            s.q, s.scale = q, 1.0
            s.k_in[..., 0] = gap
            huge = torch.arange(s.k_in.shape[0]) % 7 == 3
            s.k_in[huge, :, 0] = 0.0
            s.v_in[huge] = (s.v_in[huge].float() * 2.0 ** 110).to(s.dtype)
            s.write()
            s.check(*s.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [2, 64])
def test_keys_and_values_of_the_type_s_largest(dtype, heads):
    """Held, they stand for the next power of two, which the type has not.  A
    query that is 0 there scores as if they were not; values of it come out
    where they are not alone."""
    most = torch.finfo(DT[dtype]).max
    with Step([1, 2, 1], [40, 70, 200], [-1, 0, 0], [100], heads, 2, 64, 16, dtype, spread=0.3) as s:
        s.q = s.q.contiguous()
        s.q[..., 5] = 0
        s.k_in[::3, :, 5] = most
        s.k_in[1::3, :, 5] = -most
        s.v_in[::9, :, 7] = most
        s.v_in[1::9, :, 7] = -most
        s.write()
        s.check(*s.run())
