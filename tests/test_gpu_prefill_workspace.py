"""Workspace of the prompt's calls: what each wants for its own use, and no more."""
import pytest
import torch

import compressed_decode_attention_fdms_b200 as fd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_prefill import Call  # noqa: E402

ATTN, SCORES, KEEP = fd.FDMS_FOR_ATTN, fd.FDMS_FOR_SCORES, fd.FDMS_WITH_KEEP


def need(c, uses):
    return fd.fdms_prefill_workspace_for(c.cache, c.B, c.max_n, c.max_q, uses)


@pytest.mark.parametrize("lens,qs,rate", [([1300, 1100], None, None), ([1300, 1100], None, 0.2),
                                          ([5000], [200], None), ([5000], [200], 0.2),
                                          ([5000, 4000], [5, 3], None),
                                          ([5000, 4000], [5, 3], 0.2), ([300], None, 0.2)])
@pytest.mark.parametrize("D", [64, 128])
def test_exactly_as_much_as_is_asked_for(lens, qs, rate, D):
    """Each call with its own size, in a buffer that is watched behind it."""
    c = Call(lens, qs, 8, 2, D, W=64, rate=rate, seed=51)
    keep = 0 if rate is None else KEEP
    hold = torch.empty(max(need(c, ATTN | keep), need(c, SCORES | keep)) + 4096,
                       dtype=torch.uint8, device="cuda:0")

    def part(uses):
        hold.fill_(173)
        n = need(c, uses)
        c.ws = hold[:n]
        return n

    n = part(ATTN | keep)
    c.attn()
    torch.cuda.synchronize()
    c.check_attn()
    assert (hold[n:] == 173).all()
    n = part(SCORES | keep)
    s = c.scores(c.lse)
    torch.cuda.synchronize()
    c.check_scores(s, c.lse)
    assert (hold[n:] == 173).all()
    c.check_error()


def test_copies_of_kept_tokens_are_asked_for_where_they_are_made():
    cache = fd.fdms_cache_create(fd.make_config(1, 8, 32, 8, 128, 256, 1, 32768, 1))

    def size(max_q, uses):
        return fd.fdms_prefill_workspace_for(cache, 8, 32768, max_q, uses)

    rows = 8 * 8 * 32768 * 128 * 2               # K or V of every head
    # few rows (16 tokens x 4 heads) read the kept rows in place
    assert size(16, ATTN | KEEP) == size(16, ATTN) < rows // 16
    assert size(17, ATTN | KEEP) >= 2 * rows
    assert size(32768, ATTN) < rows // 2 and size(32768, SCORES) <= rows // 2
    assert size(32768, ATTN | KEEP) >= 2 * rows
    # scores: the K rows, a position and two bits a token, sums of both kinds of tiles
    assert rows <= size(32768, SCORES | KEEP) - 2 * size(32768, SCORES) < 1.1 * rows
    every = ATTN | SCORES | KEEP
    for max_q in (1, 17, 32768):
        sizes = [size(max_q, u) for u in range(8)]
        assert sizes[0] == sizes[KEEP] == 0
        assert max(sizes) == sizes[every] == fd.fdms_prefill_workspace(cache, 8, 32768, max_q)
    for uses in (-1, 8):
        with pytest.raises(fd.FdmsError):
            size(1, uses)


def test_refused_with_less():
    c = Call([1300], None, 8, 2, 64, W=64, rate=0.2, seed=52)
    z = torch.zeros(c.q.shape[:3], device="cuda:0")
    for uses, call in ((ATTN | KEEP, c.attn), (SCORES | KEEP, lambda: c.scores(z))):
        whole = torch.empty(need(c, uses), dtype=torch.uint8, device="cuda:0")
        c.ws = whole
        call()
        for ws in (whole[:-1], whole[:need(c, uses & ~KEEP)], None):
            c.ws = ws
            with pytest.raises(fd.FdmsError):
                call()
    torch.cuda.synchronize()
    c.check_error()


def test_larger_sizes_serve_smaller_calls():
    cache = fd.fdms_cache_create(fd.make_config(1, 8, 8, 2, 64, 64, 1, 9000, 1))
    g = torch.Generator().manual_seed(53)

    def draw(hi):
        return 1 + int(torch.randint(0, hi, (1,), generator=g))

    for _ in range(100):
        B, T = draw(8), draw(9000)
        Q = draw(T)
        b, t = draw(B), draw(T)
        q = draw(min(t, Q))
        for uses in range(8):
            size = fd.fdms_prefill_workspace_for(cache, B, T, Q, uses)
            assert fd.fdms_prefill_workspace_for(cache, b, t, q, uses) <= size
            assert fd.fdms_prefill_workspace_for(cache, B, T, Q, uses & ~KEEP) <= size
