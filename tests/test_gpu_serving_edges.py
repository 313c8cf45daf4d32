"""GPU tests of the serving operators where their answers are easiest to lose:
weights far below a head's largest, and calls that must not depend on what is
asked for beside the answer.  Plain forms and bounds: tests/serving_ref.py."""
import math

import pytest
import torch

from mass_adaptive_sparse_gb300 import api
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KEEP_ALL = 1e-30           # a tau > 0 that skips no tile of these inputs


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cuda(cache):
    return tuple(t.cuda() for t in cache)


def status():
    torch.cuda.synchronize()
    return api.mala_device_status()


# ---------------------------------------------------------------------------
# Weights far below the largest
# ---------------------------------------------------------------------------

# relative error of a weight that enters P V (fp16; fp32 queries: a sum of two), and what it is off by at most below
# that, in parts of the head's largest p * 2^e_v
U_P = {BF16: 2.0 ** -11, FP32: 2.0 ** -22}
FLOOR = {BF16: 2.0 ** -39, FP32: 2.0 ** -50}


def small_weights_limit(q, k, v, v_scale, scale, dtype):
    """The 64-bit softmax of q [G, D] over k, v [N, D], and how far an fp32 o may be from it, element by element.

    Every score here is one nonzero product, so no sum rounds in it: scale and maximum in fp32 leave
    d = 3 * 2^-24 max|s| + 2^-21 (exp2 to 2 ulp) in the exponent.  A weight p 2^e_v is off by U_P of itself, or by FLOOR
    of the largest; sums of N terms in fp32 by N 2^-24.  Numerator and denominator both carry the relative parts."""
    want, _, absv, qk = ref.attend(q, k, v, scale)
    largest = (torch.softmax((q @ k.T) * scale, -1) * v_scale).amax(-1, keepdim=True)
    codes = (v / v_scale[:, None]).abs().sum(0)
    d = (3 * 2.0 ** -24 * qk + 2.0 ** -21).unsqueeze(-1)
    limit = 2 * (d + U_P[dtype] + k.shape[0] * 2.0 ** -24) * absv + FLOOR[dtype] * largest * codes + 2.0 ** -24 * want.abs()
    return want, limit


def two_kinds_of_rows(N, D, large):
    """K and V codes (as numbers) [N, D] and value exponents: the `large` rows have key 1 in channel 0 and value 1 in the
    lower half of the channels, 0 in the upper; the others have key -1 in channel 1 and value 1.125 everywhere."""
    k, v = torch.zeros((N, D)), torch.full((N, D), 1.125)
    k[:, 1] = -1
    k[large] = 0
    k[large, 0] = 1
    v[large, :D // 2] = 1
    v[large, D // 2:] = 0
    return k, v


def as_cache(k, v, v_exps):
    """[1, N, 1, D] cache of codes k, v with scale 1 keys."""
    codes = [x[None, :, None].to(torch.float8_e4m3fn).contiguous().cuda() for x in (k, v)]
    k_exps = torch.full((1, 1, k.shape[0]), 127, dtype=torch.uint8, device="cuda")
    return codes[0], k_exps, codes[1], v_exps.to(torch.uint8).view(1, 1, -1).cuda()


@pytest.mark.parametrize("tau", [0.0, KEEP_ALL])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (FP32, 128), (FP32, 64)])
def test_decode_quant_weights_far_below_the_largest(dtype, D, tau):
    """A few keys hold nearly all of the mass, the others 2^-13 to 2^-25 of it each, and they alone have values in
    half of the channels.  Every warp meets a large key first."""
    N = 640
    large = [i for i in range(N) if i % 32 == 0 and (i < 128 or i >= 512)]
    k, v = two_kinds_of_rows(N, D, large)
    q = torch.zeros((4, D))
    q[:, 0] = torch.tensor([9.25, 12.0, 14.5, 17.25])          # nats above the others' 0
    q = q.to(dtype)
    cache = as_cache(k, v, torch.full((N,), 127))
    o, _, _ = api.decode_quant(q[None].cuda(), cache, tau, num_splits=1, softmax_scale=1.0, out_dtype=FP32)
    assert status() == 0
    want, limit = small_weights_limit(q.double(), k.double(), v.double(), torch.ones(N, dtype=torch.float64), 1.0, dtype)
    off = (o[0].double().cpu() - want).abs()
    assert (off <= limit).all(), f"off by {float((off / limit).max()):.3g} of the bound"


@pytest.mark.parametrize("ratio", [13, 20, 27, 40])
@pytest.mark.parametrize("tau", [0.0, KEEP_ALL])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
def test_decode_quant_large_rows_with_empty_channels(dtype, D, tau, ratio):
    """Value rows 2^ratio times larger than the others, but zero in half of the channels."""
    N = 640
    large = [i for i in range(N) if i % 32 == 0 and (i < 128 or i >= 512)]
    k, v = two_kinds_of_rows(N, D, large)
    q = torch.zeros((4, D))
    q[:, 1] = -torch.tensor([0.0, 0.296875, 0.546875, 0.640625])       # the small rows' scores: weights between powers of two
    q = q.to(dtype)
    exps = torch.full((N,), 127)
    exps[large] += ratio
    scale_of = torch.exp2(exps.double() - 127)
    cache = as_cache(k, v, exps)
    o, _, _ = api.decode_quant(q[None].cuda(), cache, tau, num_splits=1, softmax_scale=1.0, out_dtype=FP32)
    assert status() == 0
    v64 = v.double() * scale_of[:, None]
    want, limit = small_weights_limit(q.double(), k.double(), v64, scale_of, 1.0, dtype)
    off = (o[0].double().cpu() - want).abs()
    assert (off <= limit).all(), f"off by {float((off / limit).max()):.3g} of the bound"


# ---------------------------------------------------------------------------
# What is asked for beside the answer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tau", [0.0, 16.0])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
def test_decode_quant_counts_and_mask_do_not_change_the_answer(dtype, D, tau):
    """Without num_splits the same splits are taken, whatever is asked for beside o and lse; the counts are theirs."""
    B, N, Hkv = 3, 7000, 8             # 19 or 25 splits of three tiles on 152 multiprocessors
    host = ref.random_cache(B, N, Hkv, D, 17)
    cache = cuda(host)
    g = torch.Generator().manual_seed(23)
    near = ref.values(*host[:2])[:, 100].float()                      # queries that lean towards one key: tiles to skip
    near = near / near.square().mean(-1, keepdim=True).sqrt()
    q = (torch.randn((B, 4 * Hkv, D), generator=g) + 6 * near.repeat_interleave(4, 1)).to(dtype).cuda()
    lens = i32([N, 4999, 129])
    calls = [api.decode_quant(q, cache, tau, cache_lens=lens, counts=c, mask=m) for c, m in
             ((False, False), (True, False), (False, True), (True, True))]
    assert status() == 0
    for o, lse, _ in calls[1:]:
        assert torch.equal(o, calls[0][0]) and torch.equal(lse, calls[0][1])
    assert torch.equal(calls[1][2]["counts"], calls[3][2]["counts"]) and torch.equal(calls[2][2]["mask"], calls[3][2]["mask"])
    counts, mask = calls[3][2]["counts"].cpu(), calls[3][2]["mask"].cpu()
    splits = counts.shape[2]
    skipped = 0
    for b, n in enumerate(lens.tolist()):
        T = -(-n // 128)
        per = -(-T // splits)
        skipped += int((mask[b, :, :T] == 0).sum())
        for h in range(Hkv):
            assert counts[b, h].tolist() == [int(mask[b, h, i * per:min(T, (i + 1) * per)].sum()) for i in range(splits)]
    assert (skipped > 0) == (tau > 0)


# ---------------------------------------------------------------------------
# The skip rule where the dense passes were tested alone
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
@pytest.mark.parametrize("splits", [1, 3])
def test_decode_quant_keeps_a_tile_with_a_nan_key(dtype, D, splits):
    """A NaN score is not below the limit: its tile is kept and the answer is NaN, however small the tile's other scores are."""
    B, N, Hkv = 2, 1000, 2
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((B, N, Hkv, D), generator=g) for _ in range(2))
    q = 3 * torch.randn((B, 4 * Hkv, D), generator=g)
    tiles = 8
    per = -(-tiles // splits)
    for first in range(0, tiles, per):                                # each split's newest tile holds a key like its queries
        last = min(N, min(tiles, first + per) * 128) - 1
        k[:, last] = q[:, ::4]
    q = q[:, ::4].repeat_interleave(4, 1).to(dtype)
    k[0, 77, 1, 5] = math.nan                                         # in a tile that nothing else keeps
    cache = api.quant_cache(B, N, Hkv, D)
    api.cache_write(k.cuda(), v.cuda(), cache)
    o, lse, info = api.decode_quant(q.cuda(), cache, 1.0, num_splits=splits, mask=True)
    assert status() == 0
    mask = info["mask"].cpu()
    assert (mask[0, 0] == 0).any() and mask[1, 1, 0] == 0             # the same tile without a NaN is skipped
    assert mask[0, 1, 0] == 1
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all()
    assert torch.isfinite(lse[0, :4]).all() and torch.isfinite(lse[1]).all()


# ---------------------------------------------------------------------------
# Refusals that no allocation comes before
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("splits", [257, 10 ** 8, -10 ** 8])
def test_split_counts_out_of_range_are_refused_by_the_library(splits):
    cache = api.quant_cache(2, 16, 2, 64)
    q = torch.zeros((2, 8, 64), dtype=BF16, device="cuda")
    p = torch.zeros((5, 2, 64), dtype=BF16, device="cuda")
    for call in (lambda: api.decode_quant(q, cache, 0.0, num_splits=splits),
                 lambda: api.decode_quant(q, cache, 1.0, num_splits=splits, counts=True, mask=True),
                 lambda: api.decode_shared(q, p, p, prefix_splits=splits),
                 lambda: api.decode_shared(q, p, p, suffix_splits=splits)):
        with pytest.raises(api.MalaError) as err:
            call()
        assert err.value.code == 1
