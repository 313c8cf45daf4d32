"""GPU tests of the serving operators where their answers are easiest to lose:
weights far below a head's largest, and calls that must not depend on what is
asked for beside the answer.  Plain forms and bounds: tests/serving_ref.py."""
import math

import pytest
import torch

import oracle as orc
from mass_adaptive_sparse_gb300 import api
from tests import parity
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KEEP_ALL = 1e-30           # a tau > 0 that skips no tile whose scores lie within 69 nats of the largest


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


TAUS = [0.0, KEEP_ALL, 16.0]
U_W = {BF16: 2.0 ** -11, FP32: 2.0 ** -21}                # of the weights, as in the dense tests


def leaning_queries(B, Hq, D, dtype, seed, k, at, amp=6.0):
    """Queries that lean towards key at[b] of sequence b (k [B, N, Hkv, D], float64)."""
    g = torch.Generator().manual_seed(seed)
    near = torch.stack([k[b, at[b]] for b in range(B)]).float()
    near = near / near.square().mean(-1, keepdim=True).sqrt()
    return (torch.randn((B, Hq, D), generator=g) + amp * near.repeat_interleave(Hq // k.shape[2], 1)).to(dtype)


def check_kept(o, lse, info, q, k, v, lens, splits, tau, rows=None):
    """Decisions as the oracle's (borderline tiles replayed), counts of every head and split, and o and lse element by
    element against the 64-bit softmax over the keys of the kept tiles.  Returns the number of skipped tiles."""
    D, Hkv, dtype = q.shape[2], k.shape[2], q.dtype
    G, scale, block = q.shape[1] // Hkv, 1 / math.sqrt(D), 128
    mask, counts = info["mask"].cpu(), info["counts"].cpu()
    skipped = 0
    for b in range(q.shape[0]) if rows is None else rows:
        n = lens[b]
        T = -(-n // block)
        per = -(-T // splits)
        assert not mask[b, :, T:].any()
        for h in range(Hkv):
            kept = mask[b, h, :T] != 0
            assert counts[b, h].tolist() == [int(kept[min(T, i * per):min(T, (i + 1) * per)].sum()) for i in range(splits)]
            qh, kh, vh = q[b, h * G:(h + 1) * G].double(), k[b, :n, h], v[b, :n, h]
            want = orc.mala_decode(qh.numpy(), kh.numpy(), vh.numpy(), scale, tau, block, splits)
            parity.decode_expected(kept.numpy(), want.o, want.lse, want.retained, qh.numpy(), kh.numpy(), vh.numpy(), scale, tau,
                                   block, splits)
            skipped += int((~kept).sum())
            keys = kept.repeat_interleave(block)[:n]
            eo, el, absv, qk = ref.attend(qh, kh[keys], vh[keys], scale)
            lo, ll = ref.bounds(eo, el, absv, qk, int(keys.sum()), D, U_W[dtype], ref.U[o.dtype])
            heads = slice(h * G, (h + 1) * G)
            assert ((o[b, heads].double().cpu() - eo).abs() <= lo).all(), f"o, b={b}, h={h}"
            assert ((lse[b, heads].double().cpu() - el).abs() <= ll).all(), f"lse, b={b}, h={h}"
    return skipped


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64), (BF16, 64), (FP32, 128)])
@pytest.mark.parametrize("splits", [1, 3])
def test_decode_quant_stale_rows(dtype, D, splits, tau):
    """Rows behind the lengths hold NaN codes and the largest scales, also in tiles that a length ends in."""
    lens = [1, 31, 33, 128, 129, 900, 1023, 1100]
    B, N, Hkv, Hq = len(lens), 1100, 2, 8
    cache = ref.random_cache(B, N, Hkv, D, 121)
    k, v = (ref.values(*cache[i:i + 2]) for i in (0, 2))
    q = leaning_queries(B, Hq, D, dtype, 14, k, [n - 1 for n in lens])
    for b, n in enumerate(lens):
        for i in (0, 2):
            cache[i].view(torch.uint8)[b, n:] = 0x7f
            cache[i + 1][b, :, n:] = 255 if b % 2 else 254
    o, lse, info = api.decode_quant(q.cuda(), cuda(cache), tau, num_splits=splits, cache_lens=i32(lens), counts=True, mask=True)
    assert status() == 0
    skipped = check_kept(o, lse, info, q, k, v, lens, splits, tau)
    assert skipped == 0 if tau == 0 else skipped > 0 or tau == KEEP_ALL


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
def test_decode_quant_wrong_lengths_at_every_tau(dtype, D, tau):
    """A refused length gives NaN, no kept tile and the status bit; the sequences beside it are answered."""
    lens, N = [500, 0, 700, -3, 701, 1], 700
    B, Hkv, Hq, splits = len(lens), 2, 8, 2
    cache = ref.random_cache(B, N, Hkv, D, 12)
    k, v = (ref.values(*cache[i:i + 2]) for i in (0, 2))
    good = [b for b, n in enumerate(lens) if 1 <= n <= N]
    q = leaning_queries(B, Hq, D, dtype, 15, k, [n - 1 if b in good else 0 for b, n in enumerate(lens)])
    o, lse, info = api.decode_quant(q.cuda(), cuda(cache), tau, num_splits=splits, cache_lens=i32(lens), counts=True, mask=True)
    assert status() == 2
    for b in range(B):
        if b not in good:
            assert torch.isnan(o[b]).all() and torch.isnan(lse[b]).all()
            assert not info["counts"][b].any() and not info["mask"][b].any()
    check_kept(o, lse, info, q, k, v, lens, splits, tau, rows=good)


@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_quant_nonfinite_rows_and_queries(dtype, tau):
    """A NaN key makes its KV head's answers NaN, an infinite value row those that weigh it, a NaN query its own head's."""
    B, N, Hkv, Hq, D = 3, 700, 2, 8, 128
    g = torch.Generator().manual_seed(33)
    k, v = (torch.randn((B, N, Hkv, D), generator=g) for _ in range(2))
    q = torch.randn((B, Hq, D), generator=g).to(dtype)
    k[0, 77, 1, 5] = math.nan
    v[1, N - 1, 0, 9] = -math.inf                      # in the newest tile, which is always kept
    q[2, 3, 0] = math.nan
    cache = api.quant_cache(B, N, Hkv, D)
    api.cache_write(k.cuda(), v.cuda(), cache)
    o, lse, _ = api.decode_quant(q.cuda(), cache, tau, num_splits=1)
    assert status() == 0
    bad_o = torch.zeros((B, Hq), dtype=torch.bool)
    bad_o[0, 4:] = bad_o[1, :4] = bad_o[2, 3] = True
    bad_lse = bad_o.clone()
    bad_lse[1] = False                                 # values do not enter it
    assert torch.equal(torch.isnan(o).all(-1).cpu(), bad_o) and torch.equal(torch.isnan(o).any(-1).cpu(), bad_o)
    assert torch.equal(torch.isnan(lse).cpu(), bad_lse)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
def test_decode_quant_same_bits_under_the_skip_rule(dtype, D):
    cache = ref.random_cache(3, 3000, 4, D, 181)
    q = leaning_queries(3, 16, D, dtype, 3, ref.values(*cache[:2]), [2999, 10, 1500]).cuda()
    cache = cuda(cache)
    a, b = (api.decode_quant(q, cache, 16.0, num_splits=3, cache_lens=i32([3000, 2999, 130]), counts=True, mask=True) for _ in range(2))
    assert status() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(a[2][n], b[2][n]) for n in ("counts", "mask"))


@pytest.mark.parametrize("tau", [KEEP_ALL, 1.0])
def test_skip_rule_offsets_past_32_bits(tau):
    """A cache whose last rows lie more than 2^31 bytes in, under the skip rule: decisions are not replayed here, but o and lse
    are the softmax over the keys of the tiles that the mask names, the newest among them."""
    N, Hkv, D, splits = 2_200_000, 8, 128, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = [torch.empty((1, N, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.full((1, Hkv, N), 122, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for c in codes:
        for i in range(0, N, 200_000):
            c[:, i:i + 200_000] = torch.randn((1, min(200_000, N - i), Hkv, D), generator=g, device="cuda").mul_(32).to(torch.float8_e4m3fn)
    q = torch.randn((1, 16, D), generator=g, device="cuda").to(BF16)
    q[:, 14:] += 6 * codes[0][:, N - 1, 7:8].to(torch.float32).sign().to(BF16)   # the last head's queries lean towards the last row
    o, lse, info = api.decode_quant(q, (codes[0], exps[0], codes[1], exps[1]), tau, num_splits=splits, counts=True, mask=True)
    assert status() == 0
    kept = info["mask"][0, 7] != 0
    T = kept.numel()
    per = -(-T // splits)
    assert info["counts"][0, 7].tolist() == [int(kept[i * per:(i + 1) * per].sum()) for i in range(splits)]
    assert bool(kept[-1]) and bool(kept.all()) == (tau == KEEP_ALL)
    keys = kept.repeat_interleave(128)[:N]
    rows = [(codes[i][0, :, 7][keys].double() * torch.exp2(exps[i][0, 7][keys].double() - 127)[:, None]) for i in (0, 1)]
    want_o, want_lse, absv, qk = ref.attend(q[0, 14:].double(), rows[0], rows[1], 1 / math.sqrt(D))
    lo, ll = ref.bounds(want_o, want_lse, absv, qk, int(keys.sum()), D, U_W[BF16], ref.U[BF16])
    assert ((o[0, 14:].double() - want_o).abs() <= lo).all() and ((lse[0, 14:].double() - want_lse).abs() <= ll).all()


def test_raw_calls_refuse_missing_outputs():
    """The entry points that return nothing take their outputs from the caller: None is not a place to drop a result."""
    cache = api.quant_cache(2, 16, 2, 64)
    q = torch.zeros((2, 8, 64), dtype=BF16, device="cuda")
    p = torch.zeros((5, 2, 64), dtype=BF16, device="cuda")
    lse = torch.zeros((2, 8), device="cuda")
    launched = api.mala_launch_count()
    for o, l, name in ((None, lse, "o"), (q.clone(), None, "lse"), (None, None, "o")):
        with pytest.raises(ValueError, match=f"{name} must be a tensor"):
            api.mala_decode_quant(q, *cache, o, l, None)
        with pytest.raises(ValueError, match=f"{name} must be a tensor"):
            api.mala_decode_shared(q, p, p, None, None, o, l, None)
    with pytest.raises(ValueError, match="k must be a tensor"):
        api.mala_cache_read(*cache, None, None)
    assert api.mala_launch_count() == launched
