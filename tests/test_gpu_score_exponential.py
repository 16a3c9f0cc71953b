"""The exponentials of the scores (four columns of sixteen by a polynomial, the others
by the special-function unit), one at a time, against 64 bits."""
import numpy as np
import pytest
import torch

import compressed_decode_attention_fdms_b200 as fd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

# The polynomial: 7.5e-8 for its degree (ln(2)^6 / 2^6 / 6! / 2^5, 1.3 * 2^-24) over values
# of 0.7 or more, at most 1.8 * 2^-24 relative, and 2^-24 and less for the last fp32 step
# and a third of it for the one before: under 4 * 2^-24. The unit: its documented 2^-22.
REL = 2.0 ** -22
LEAST = 2.0 ** -126                  # results under it may be 0


@pytest.mark.parametrize("column", [0, 1, 2, 3, 4, 9, 15, 64, 67, 112, 127])
def test_one_weight(column):
    """128 queries after T tokens, all but one with a denominator of +inf (weights of 0):
    token j's score is 2^x_j for that one, x_j = k_j log2(e) - lse log2(e)."""
    T = 4096
    n = T + 128
    cache = fd.fdms_cache_create(fd.make_config(1, 1, 1, 1, 64, n, 1, n, 1, "bf16", 1.0))
    g = torch.Generator().manual_seed(column)
    k = torch.zeros((1, n, 1, 64))
    k[0, :, 0, 0] = torch.rand(n, generator=g) * 176.0 - 88.0
    k[0, :64, 0, 0] = torch.linspace(-92.0, 92.0, 64)        # past either end
    k = k.bfloat16()
    q = torch.zeros((1, 128, 1, 64)).bfloat16()
    q[..., 0] = 1.0
    for z in (0.0, 0.37, -0.8125, 3.3):
        lse = torch.full((1, 128, 1), float("inf"), device="cuda:0")
        lse[0, column] = z
        scores = torch.zeros((1, 1, n), device="cuda:0")
        ws = torch.empty(max(1, fd.fdms_prefill_workspace(cache, 1, n, 128)), dtype=torch.uint8,
                         device="cuda:0")
        fd.fdms_prefill_scores(cache, 1, torch.tensor([n], dtype=torch.int32, device="cuda:0"), n,
                               q.cuda(), k.cuda(), lse, scores,
                               nq=torch.tensor([128], dtype=torch.int32, device="cuda:0"),
                               workspace=ws)
        got = scores[0, 0, :T].cpu().double().numpy()
        # the exponent as fp32 holds it: one rounding of a product and a sum
        log2e = np.float32(1.4426950408889634)
        off = np.float32(np.float32(z) * -log2e)
        s = k[0, :T, 0, 0].double().numpy()
        x = (s * np.float64(log2e) + np.float64(off)).astype(np.float32).astype(np.float64)
        want = np.exp2(x)
        inside = x < 127.0
        assert (np.abs(got - want) <= REL * want + LEAST)[inside].all(), \
            (z, np.abs(got / want - 1)[inside & (want > LEAST)].max())
        assert (got[x < -127.0] == 0).all()
        assert (np.isinf(got) | (np.abs(got - want) <= REL * want))[~inside].all()
        assert (got[~inside] >= 2.0 ** 126.9).all()
    assert fd.fdms_cache_stats(cache)["error"] == 0
