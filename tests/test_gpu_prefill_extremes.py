"""Prompt attention where the parts of a row's keys differ by all that fp32 holds:
splits whose sums come from a late jump."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_prefill import Call, both  # noqa: E402


@pytest.mark.parametrize("first,second", [(660, 660), (696, 704), (700, 700), (704, 700),
                                          (708, 708), (716, 716)])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 2)])
@pytest.mark.parametrize("rate", [None, 1.0])
def test_jumps_on_both_sides_of_a_split(first, second, D, G, rate):
    """32 key tiles in eight runs of four (with kept tokens: 33). Tokens 511 and 512,
    the last of the first run and the first of the second, have scores of 82.5 to 89.5
    (119 to 129 bits), all others 0: each of the two carries a share of every row.
    Values are small, so that no sum of the first five overflows."""
    c = Call([4096], [200], G, 1, D, W=4096 if rate is None else 64, rate=rate, seed=41,
             scale=0.125)
    c.q[:], c.k[:] = 0.0, 0.0
    c.q[..., 0] = 1.0
    c.k[0, 511, 0, 0], c.k[0, 512, 0, 0] = first, second
    c.v *= 2.0 ** -8
    both(c)
