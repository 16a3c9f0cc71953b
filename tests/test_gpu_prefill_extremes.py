"""Prompt attention where the parts of a row's keys differ by all that fp32 holds:
splits whose sums come from a late jump, rows computed a second time whose first
key has a score of -inf, values near the end of the range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from _prompt import f64  # noqa: E402
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


@pytest.mark.parametrize("T,qs", [(300, None), (700, None), (1100, None), (700, [5])])
@pytest.mark.parametrize("D", [64, 128])
def test_first_key_of_minus_infinity_in_rows_computed_again(T, qs, D):
    """Token 0, which every row sees, has a score of -inf: a weight of 0. A V row
    that the last rows do not see, but others of their tile do, holds infinities, so
    that they are computed again, from token 0 on."""
    W, gone = 2, T - 5
    c = Call([T], qs, 4, 2, D, W=W, rate=0.3, seed=42)
    c.keep[0, 0] = 1
    c.keep[0, gone] = 0
    c.q[..., 0] = 1.0
    c.k[0, 0, :, 0] = float("-inf")
    c.v[0, gone] = float("inf")
    c.attn()
    torch.cuda.synchronize()
    rows = slice(T - 3, T) if qs is None else slice(2, 5)   # tokens T - 3 and later
    # those rows' results are what they are without tokens 0 and `gone`
    c.keep[0, 0] = 0
    c.k[0, 0, :, 0] = 0.0
    c.v[0, gone] = 0.0
    o, z, tol, ztol = (x[rows] for x in c.reference(0))
    assert (np.abs(f64(c.out)[0, rows] - o) <= tol).all()
    assert (np.abs(f64(c.lse)[0, rows] - z) <= ztol).all()
    c.check_error()


@pytest.mark.parametrize("T,qs", [(300, None), (700, None), (2100, [7])])
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_end_of_the_range(T, qs, D):
    """Sums of V rows pass what fp32 holds, their weighted means do not."""
    c = Call([T], qs, 4, 2, D, W=T, seed=43, spread=0.2)
    c.v[..., 1] = 2.0 ** 127
    c.v[..., 2] = -(2.0 ** 126)
    c.v[:, ::2, :, 3] = 2.0 ** 127
    c.v[:, 1::2, :, 3] = -(2.0 ** 127)
    c.attn()
    torch.cuda.synchronize()
    c.check_attn()
    c.check_error()
