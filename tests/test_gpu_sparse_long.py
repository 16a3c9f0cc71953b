"""Block-sparse decode over stores whose blocks several CTAs score (32 each) and
rank in more than one round (256 each): the last one's hand-over, the count that
starts again at 0, bounds found by several CTAs, exact ranks, and stores whose
scores are not kept in shared memory."""
import pytest
import torch

import compressed_decode_attention_fdms_b200 as fd

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from _prompt import dev  # noqa: E402
from test_gpu_sparse import KV, Sparse  # noqa: E402

W = 24


def tokens(full):
    """Of a context that keeps everything and has `full` full blocks and 40 slots more."""
    return full * 64 + 40 + W


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("full", [32, 33, 64, 65, 257])
def test_blocks_of_several_ctas(kv, full):
    """The second sequence has fewer blocks than the first (and fewer CTAs)."""
    s = Sparse([tokens(full), tokens(full // 3)], 4, 2, 64, W=W, rate=1.0, kv=kv, seed=61)
    fd.fdms_bounds_create(s.cache)
    s.check(5)
    s.check(5, q=-s.q)
    s.check(full - 1)
    for t in range(30):                  # 24 tokens on, the partly filled block is full
        s.step(0, 6100 + t)
        if t % 7 == 0:
            s.decode(5, blocks=False)
    s.check(5)
    s.check(full)
    s.check(full + 1)


@pytest.mark.parametrize("heads", [(8, 1, 128), (3, 3, 128)])
def test_heads_of_different_lengths(heads):
    s = Sparse([9000, 5000, 2500], *heads, W=W, rate=0.7, seed=62)
    fd.fdms_bounds_create(s.cache)
    for num in (1, 7, 50):
        s.check(num)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3_block"])
def test_six_hundred_blocks(kv):
    s = Sparse([tokens(600)], 2, 1, 64, W=W, rate=1.0, kv=kv, seed=63)
    fd.fdms_bounds_create(s.cache)
    s.check(32)
    s.check(300)


def test_first_call_after_many_dense_ones():
    """Bounds of all blocks at once, after steps that needed none."""
    s = Sparse([tokens(70)], 4, 2, 64, W=W, rate=1.0, seed=64)
    fd.fdms_bounds_create(s.cache)
    out = torch.empty(s.q.shape, dtype=torch.bfloat16, device="cuda:0")
    for t in range(40):
        s.step(0, 6400 + t)
        fd.fdms_decode_attn(s.cache, 0, 1, dev(s.q), out)
    s.decode(1000)                       # as many blocks as there are: no bounds needed
    s.check(3)


def filled(k, room=100):
    """A cache of one sequence and head pair that keeps the rows k [T][64] of both heads."""
    T = k.shape[0]
    s = Sparse([1], 4, 2, 64, W=0, rate=1.0, seed=65, room=T + room)
    v = torch.randn((1, T, 2, 64), generator=torch.Generator().manual_seed(66)).bfloat16()
    s.append(0, k[None, :, None, :].expand(1, T, 2, 64), v,
             torch.ones((1, T, 2), dtype=torch.uint8), [T])
    fd.fdms_bounds_create(s.cache)
    return s


def test_equal_scores_past_one_round():
    """A token in front: block j holds the rows 64 j - 1 .. 64 j + 62 of k."""
    k = torch.ones((64 * 400, 64)).bfloat16()
    for j in (3, 255, 256, 257, 300, 390):
        k[64 * j + 10] = 2.0
    s = filled(k)
    s.q = torch.ones((1, 4, 64)).bfloat16()
    for num in (1, 4, 6, 7, 260, 399):
        s.check(num)
    s.check(5, q=-s.q)
    s.check(300, q=0 * s.q)


@pytest.mark.parametrize("down", [False, True])
def test_scores_that_fp32_cannot_tell_apart(down):
    """Scores of 4096 + j 2^-16: exact in the kernel's sums, equal in fp32."""
    k = torch.zeros((64 * 270, 64)).bfloat16()
    k[:, 0] = 4096.0
    j = torch.arange(64 * 270) // 64
    k[:, 9] = (torch.where(j < 256, j, 600 - 2 * j) * (-1.0 if down else 1.0) *
               2.0 ** -16).bfloat16()
    s = filled(k)
    s.q = torch.zeros((1, 4, 64)).bfloat16()
    s.q[..., 0] = 1.0
    s.q[..., 9] = 1.0
    for num in (1, 17, 200):
        s.check(num)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("full", [20, 70, 300])
def test_scores_not_in_shared_memory(kv, full):
    """A cache with room for more blocks (3,600 and more) than the shared memory of a
    CTA takes scores of."""
    s = Sparse([tokens(full)], 2, 1, 64, W=W, rate=1.0, kv=kv, seed=67, room=64 * 3700)
    fd.fdms_bounds_create(s.cache)
    s.check(5)
    s.check(5, q=-s.q)
    for t in range(30):
        s.step(0, 6700 + t)
    s.check(17)


@pytest.mark.parametrize("first,second", [(float("nan"), float("inf")),
                                          (float("inf"), float("nan"))])
def test_scores_of_infinity_and_nan_tie(first, second):
    k = torch.randn((64 * 50, 64), generator=torch.Generator().manual_seed(68)).bfloat16()
    k[64 * 7 + 5, 3] = first
    k[64 * 40 + 5, 3] = second
    s = filled(k)
    s.q = torch.ones((1, 4, 64)).bfloat16()
    for num, want in ((1, [7]), (2, [7, 40])):
        _, ids = s.decode(num)
        torch.cuda.synchronize()
        assert ids[0].tolist() == [want, want]
    assert fd.fdms_cache_stats(s.cache)["error"] == 0


def test_two_caches_in_turn():
    """Each cache has its own counts and bounds; calls on both, on two streams."""
    a = Sparse([tokens(65)], 4, 2, 64, W=W, rate=1.0, seed=69)
    b = Sparse([tokens(40), tokens(90)], 4, 2, 64, W=W, rate=1.0, seed=70)
    for s in (a, b):
        fd.fdms_bounds_create(s.cache)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(s1):
            ra = a.decode(6)
        with torch.cuda.stream(s2):
            rb = b.decode(9)
    torch.cuda.synchronize()
    a.check(6, result=ra)
    b.check(9, result=rb)


def test_rows_are_read_once_each():
    """Counters: the chosen blocks, the partly filled one and the ring."""
    s = Sparse([tokens(130)], 4, 2, 64, W=W, rate=1.0, seed=71)
    fd.fdms_bounds_create(s.cache)
    before = fd.fdms_cache_stats(s.cache)
    s.decode(12)
    after = fd.fdms_cache_stats(s.cache)
    assert after["slots_decoded"] - before["slots_decoded"] == 2 * (12 * 64 + 40 + W)
    assert after["bytes_decoded"] - before["bytes_decoded"] == \
        2 * (12 * 64 + 40 + W) * 2 * 64 * 2
