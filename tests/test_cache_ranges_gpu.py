"""Decodes over the bounded cache at the ends of their range: queries, scales and rows of any finite size, and rows of values of unlike size.

Each result is held against 64 bits within what its roundings add up to.  A score is a sum of d products that the tensor cores
take 16 at a time: counted as one unit, 2^-23 of |q|_2 |k|_2 |scale|, per step and eight for what comes after, it is off by at
most delta = (d / 16 + 8) 2^-23 |q|_2 |k|_2 |scale|.  The LSE is off by the mean of its keys' deltas by weight, and by
2^-20 (1 + |LSE|) for its own exponentials and logarithm; a weight exp(score - LSE) by a factor 1 +- rel, rel the sum of both.
A weight enters the sum of values rounded to 12 bits with its row's scale (4-bit caches) or as two bf16 parts (16 bits), and
the output is rounded to bf16 (half a step: 2^-8).
"""
import math

import pytest
from test_cache_gpu import i32, random_cache, rnd, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa(cuda_device):
    import memory_optimal_sdpa_b200 as m
    yield m
    assert m.get_last_device_error() == m.SDPA_OK


def values_abs64(codes, scales):
    """s c + |m|: what the products of a 4-bit row add up to before signs cancel."""
    s = scales.clone()
    s[..., 1] = s[..., 1].abs()
    return values64(codes, s)


def check(sdpa, q, cache, lens, scale, acc=None):
    """One decode over `cache` (4-bit, or a pair of bf16 tensors) against 64 bits, head by head."""
    import torch
    bits4 = len(cache) == 4
    if bits4:
        k, v = values64(cache[0], cache[1]), values64(cache[2], cache[3])
        k_abs, v_abs = values_abs64(cache[0], cache[1]), values_abs64(cache[2], cache[3])
    else:
        k, v = cache[0].double(), cache[1].double()
        k_abs, v_abs = k.abs(), v.abs()
    B, Hkv, cap, d = k.shape
    G = q.shape[1] // Hkv
    acc = torch.zeros((B, Hkv, cap), device="cuda") if acc is None else acc
    call = sdpa.decode_kv4(q, sdpa.Kv4Cache(*cache), i32(lens), scale=scale, acc=acc) if bits4 else sdpa.decode_acc(q, *cache, i32(lens), acc, scale=scale)
    O, L = (t.double().view(B, Hkv, G, -1) for t in call)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            qq = q[b].double().view(Hkv, G, d)[h]
            s = qq @ k[b, h, :n].T * scale
            lse = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            # per key; the LSE is off by what its keys' scores are, weighted
            delta = (d / 16 + 8) * 2.0 ** -23 * qq.norm(dim=-1)[:, None] * k_abs[b, h, :n].norm(dim=-1) * abs(scale)
            of_lse = (p * delta).sum(-1, keepdim=True) + 2.0 ** -20 * (1 + lse[:, None].abs())
            rel = delta + of_lse
            assert (p * rel).sum(-1).max() < 0.02  # the inputs leave something to check
            assert ((L[b, h] - lse[:, None]).abs() <= of_lse).all(), (b, h)
            want = p @ v[b, h, :n]
            allowed = 2.0 ** -8 * want.abs() + (p * ((2.0 ** -12 if bits4 else 2.0 ** -17) + rel)) @ v_abs[b, h, :n] + 2.0 ** -126
            assert ((O[b, h] - want).abs() <= allowed).all(), (b, h, ((O[b, h] - want).abs() / allowed).max().item())
            # a weight below 2^-126 is not a normal 32-bit number
            assert ((acc[b, h, :n].double() - p.sum(0)).abs() <= (rel * p).sum(0) + 2.0 ** -22 * p.sum(0) + G * 2.0 ** -126).all()


def scaled(cache, which, factor):
    """A cache whose keys or values are `factor` (a power of two) times as large."""
    cache = list(cache)
    at = {"k": 0, "v": 1}[which]
    at = 2 * at + 1 if len(cache) == 4 else at
    cache[at] = (cache[at].double() * factor).to(cache[at].dtype)
    return cache


def make(sdpa, bits, B, Hkv, cap, d, lens, seed):
    if bits == 4:
        return list(random_cache(sdpa, B, Hkv, cap, d, lens, seed))
    return [rnd((B, Hkv, cap, d), seed), rnd((B, Hkv, cap, d), seed + 1)]


# ------------------------------------------------------------------------------------------ sizes of q, of the scale and of the keys
# The largest element of a head is in [2^e, 2^(e + 1)), scale is 2^a / 8, keys are times 2^b; e + a + b = 0 but for the last.
EXPONENTS = [(127, -124, 0), (126, -123, 0), (125, -125, 0), (120, 0, -120), (127, -7, -120), (110, 10, -120), (124, -124, 0), (60, -60, 0),
             (-60, 60, 0), (-100, 100, 0), (-120, 120, 0), (-126, 126, 0), (-126, 66, 60), (-20, -100, 120), (-126, 6, 120), (127, -127, -3),
             (103, -138, 35), (60, -140, 80), (127, -146, 19)]


@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (128, 12)])
@pytest.mark.parametrize("e,a,b", EXPONENTS)
@pytest.mark.parametrize("bits", [4, 16])
def test_size_of_queries_scale_and_keys(sdpa, bits, e, a, b, d, G):
    import torch
    q = rnd((1, G, d), 1).double()
    if bits == 16 and e + b > 115:
        pytest.skip("the product q k is beyond 32 bits")
    top = q.abs().amax(-1, keepdim=True)
    q = (q / top * 1.5 * 2.0 ** e).to(torch.bfloat16)
    cache = scaled(make(sdpa, bits, 1, 1, 150, d, [150], 2), "k", 2.0 ** b)
    scale = 2.0 ** a / 8
    assert torch.isfinite(q).all()
    check(sdpa, q, cache, [150], scale)
    check(sdpa, q, cache, [150], -scale)


@pytest.mark.parametrize("bits", [4, 16])
def test_heads_of_unlike_size(sdpa, bits):
    """Each head has a factor of its own; one with a score that counts beside others that are far from it."""
    import torch
    d, sizes = 64, [127, 120, 100, 3, 0, -20, -126, 125] if bits == 4 else [115, 108, 88, 3, 0, -20, -126, 113]
    q = rnd((1, 8, d), 1).double()
    q = (q / q.abs().amax(-1, keepdim=True) * 1.5 * 2.0 ** torch.tensor(sizes, device="cuda")[:, None].double()).to(torch.bfloat16)
    check(sdpa, q, make(sdpa, bits, 1, 1, 97, d, [97], 2), [97], 2.0 ** -max(sizes))


@pytest.mark.parametrize("scale", [2.0 ** 127, 1.4765625 * 2.0 ** 127, (2 - 2.0 ** -23) * 2.0 ** 127, -(2 - 2.0 ** -23) * 2.0 ** 127])
@pytest.mark.parametrize("bits", [4, 16])
def test_largest_scales(sdpa, bits, scale):
    """scale log2 e may be beyond the largest 32-bit number: scores of 0 are 0, and small ones are what they are."""
    import torch
    d, n = 64, 100
    q, k = torch.zeros((1, 2, d), device="cuda"), torch.zeros((1, 1, n, d), device="cuda")
    q[0, 0, 5], q[0, 1, 37] = 2.0 ** -63, -(2.0 ** -62)
    k[..., 5], k[..., 37] = 2.0 ** -63 * (torch.arange(n) % 7 - 3), 2.0 ** -63 * (torch.arange(n) % 3)
    v = rnd((1, 1, n, d), 3)
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    if bits == 4:
        cache = sdpa.kv4_cache(1, 1, n, d)
        sdpa.kv4_append(cache, k, v, i32([0]))
        # the groups' codes give these keys back exactly, or nearly: what the cache stands for counts
        check(sdpa, q, list(cache), [n], scale)
    else:
        check(sdpa, q, [k, v], [n], scale)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, -(2.0 ** -140)])
def test_scale_of_nothing_with_huge_keys(sdpa, bits, scale):
    """A scale of 0 (or next to it) gives every key the same weight, however large its products are."""
    import torch
    d, n = 64, 80
    cache = scaled(make(sdpa, bits, 1, 1, n, d, [n], 5), "k", 2.0 ** 100)
    q = (rnd((1, 3, d), 6).double() * 2.0 ** 17).to(torch.bfloat16)
    check(sdpa, q, cache, [n], scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv,causal", [(128, 256, False), (300, 300, True), (5, 64, True)])
@pytest.mark.parametrize("scale", [2.0 ** 126, (2 - 2.0 ** -23) * 2.0 ** 127, -(2 - 2.0 ** -23) * 2.0 ** 127])
def test_prompt_weights_of_the_largest_scales(sdpa, scale, n_q, n_kv, causal, d):
    import torch
    q, k = torch.zeros((1, 2, n_q, d), device="cuda"), torch.zeros((1, 1, n_kv, d), device="cuda")
    q[0, 0, :, 5], q[0, 1, :, 37] = 2.0 ** -63 * (torch.arange(n_q) % 3), -(2.0 ** -62)
    k[..., 5], k[..., 37] = 2.0 ** -63 * (torch.arange(n_kv) % 7 - 3), 2.0 ** -63 * (torch.arange(n_kv) % 3)
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    s = q.double() @ k.double().transpose(-1, -2) * scale
    if causal:
        s.masked_fill_(torch.arange(n_kv, device="cuda") > torch.arange(n_q, device="cuda")[:, None] + (n_kv - n_q), -torch.inf)
    lse = torch.logsumexp(s, -1).float()
    want = torch.exp(s - lse[..., None].double()).sum((1, 2))
    acc = sdpa.fwd_acc(q, k, lse, causal=causal, scale=scale)
    # products of powers of two with one to three, exact; the exponents round at 2^-24 of |score| + |LSE| < 32, and the sums as in other cases
    rel = 32 * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * (2 * n_q) ** 0.5
    assert ((acc.double()[:, 0] - want).abs() <= rel * want + 2 * n_q * 2.0 ** -126).all()


# ------------------------------------------------------------------------------------------ keys that count nothing
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 12])
@pytest.mark.parametrize("lo,hi", [(0, 64), (0, 200), (64, 128), (100, 300), (0, 700), (640, 700), (0, 699), (1, 700)])
def test_keys_of_minus_infinity(sdpa, d, G, lo, hi):
    """Keys lo .. hi - 1 score -inf with every head of a group: they weigh 0, and nothing else changes.  Where they are all the keys
    there are, O = 0, LSE = -inf and every weight is 0, as for a sequence of length 0."""
    import torch
    n, Hkv = 700, 2
    q, k, v = rnd((2, Hkv * G, d), 1), rnd((2, Hkv, n + 3, d), 2), rnd((2, Hkv, n + 3, d), 3)
    q[..., 5] = q[..., 5].abs() + 0.5
    k[0, 1, lo:hi, 5] = -math.inf
    acc = torch.zeros((2, Hkv, n + 3), device="cuda")
    O, L = sdpa.decode_acc(q, k, v, i32([n, n]), acc)
    rest = [j for j in range(n) if not lo <= j < hi]
    assert torch.isfinite(O).all() and (acc[0, 1, lo:hi] == 0).all()
    if rest:
        short = torch.zeros((1, 1, len(rest)), device="cuda")
        heads = slice(G, 2 * G)
        o, l = sdpa.decode_acc(q[:1, heads].contiguous(), k[:1, 1:, rest].contiguous(), v[:1, 1:, rest].contiguous(), i32([len(rest)]), short)
        # the same keys in another order of summation
        assert torch.allclose(O[:1, heads].float(), o.float(), rtol=2.0 ** -6, atol=2.0 ** -10) and torch.allclose(L[:1, heads], l, rtol=0, atol=1e-4)
        assert torch.allclose(acc[0, 1, rest], short[0, 0], rtol=2e-4, atol=0)
    else:
        assert (O[0, G:] == 0).all() and (L[0, G:] == -math.inf).all()
    plain = torch.zeros_like(acc)
    k[0, 1, lo:hi, 5] = 0
    O2, L2 = sdpa.decode_acc(q, k, v, i32([n, n]), plain)
    others = [(0, 0), (1, 0), (1, 1)]
    for b, h in others:
        at = slice(h * G, h * G + G)
        assert torch.equal(O[b, at], O2[b, at]) and torch.equal(L[b, at], L2[b, at]) and torch.equal(acc[b, h], plain[b, h])


# ------------------------------------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("size", [2, 10, 17, 20, 21, 24, 28, 31, 33, 60, 100, 125])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("bits", [4, 16])
def test_scores_of_any_size(sdpa, bits, G, sign, size):
    """Scores of up to 2^size, exact in 32 bits: two keys, in two places, share the largest.  Their weights are a half where it is far
    above the rest, however large it is."""
    import torch
    d, n = 64, 300
    q = torch.full((1, G, d), 2.0 ** (size - 6), device="cuda").to(torch.bfloat16)
    t = (torch.arange(n) % 13 - 8) / 8.0
    t[17] = t[200] = 1.0
    t = t * 2.0 if sign > 0 else (t - 2.0) * 2.0  # the largest: 2, or -2
    k = t.to("cuda")[:, None].expand(n, d).to(torch.bfloat16).view(1, 1, n, d).contiguous()
    v = rnd((1, 1, n, d), 3)
    acc = torch.zeros((1, 1, n), device="cuda")
    if bits == 4:
        cache = sdpa.kv4_cache(1, 1, n, d)
        sdpa.kv4_append(cache, k, v, i32([0]))
        v64 = values64(cache.v_codes, cache.v_scales)[0, 0]
        O, L = sdpa.decode_kv4(q, cache, i32([n]), scale=0.5, acc=acc)
    else:
        v64 = v[0, 0].double()
        O, L = sdpa.decode_acc(q, k, v, i32([n]), acc, scale=0.5)
    s = q[0].double() @ k[0, 0].double().T * 0.5
    p, lse = torch.softmax(s, -1), torch.logsumexp(s, -1)
    # a score is exact but for the rounding of scale log2 e; weights that count differ by less than 2^7 in their scores
    assert ((acc[0, 0].double() - p.sum(0)).abs() <= 2.0 ** -14 * p.sum(0) + G * 2.0 ** -126).all()
    assert ((L[0].double() - lse).abs() <= 2.0 ** -21 * (1 + lse.abs())).all()
    want, size_of = p @ v64, p @ v64.abs()
    # 4 bits: a value is s c + m; its parts are at most 16 times as large
    assert ((O[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -12 * 16 if bits == 4 else 2.0 ** -12) * size_of).all()


@pytest.mark.parametrize("lo,hi", [(0, 128), (128, 384), (0, 511), (0, 512)])
def test_scores_below_the_range_in_4_bits(sdpa, lo, hi):
    """Keys whose products are below the least 32-bit number count nothing; without others the outputs are 0 and the LSE -inf."""
    import torch
    d, n, G = 128, 512, 4
    cache = make(sdpa, 4, 1, 1, n, d, [n], 4)
    q = (rnd((1, G, d), 5).abs().double() * 2.0 ** 60 + 2.0 ** 60).to(torch.bfloat16)
    scale = 2.0 ** -62
    cache[1][0, 0, lo:hi, :, 0], cache[1][0, 0, lo:hi, :, 1] = 0.0, -(2.0 ** 120)  # scores of -2^125 or so times 1.44, and of less
    q[0, 1] = q[0, 1] * 2.0 ** 60
    acc = torch.zeros((1, 1, n), device="cuda")
    O, L = sdpa.decode_kv4(q, sdpa.Kv4Cache(*cache), i32([n]), scale=scale, acc=acc)
    k, v = values64(cache[0], cache[1])[0, 0], values64(cache[2], cache[3])[0, 0]
    head = 1  # its scores: |q| = 2^120, -2^120 keys: below -2^128 in 32 bits
    s = q[0].double() @ k.T * scale
    if hi - lo < n:
        p = torch.softmax(s, -1)
        assert torch.isfinite(O).all() and torch.isfinite(L).all() and torch.isfinite(acc).all() and (acc[0, 0, lo:hi] == 0).all()
        rest = [j for j in range(n) if not lo <= j < hi]
        big = int(s[head, rest].argmax())
        assert p[head, rest[big]] > 0.999  # with q this large one key has it all
        assert torch.allclose(O[0, head].double(), v[rest[big]], rtol=2.0 ** -7, atol=1e-6)
    else:
        assert (O[0, head] == 0).all() and L[0, head] == -math.inf


# ------------------------------------------------------------------------------------------ values of unlike size
@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 20, 2.0 ** 24, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("at", [(0,), (3,), (40,), (149,), (0, 33, 64, 96), (5, 6, 7, 8, 9, 10, 149)])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (64, 12)])
def test_values_of_a_key_that_counts_nothing(sdpa, d, G, ratio, at):
    """Values `ratio` times as large as the others', with a weight of (nearly) 0, leave the other keys' as exact as they were."""
    import torch
    cache = make(sdpa, 4, 1, 1, 150, d, [150], 7)
    q = rnd((1, G, d), 8)
    q[..., 0] = q[..., 0].abs() + 2
    for j in at:  # -960 in channel 0, else 0: far below every other score
        cache[0][0, 0, j] = 255
        cache[0][0, 0, j, 0] = 240
        cache[1][0, 0, j] = 0
        cache[1][0, 0, j, 0, 0], cache[1][0, 0, j, 0, 1] = 64.0, -960.0
        cache[3][0, 0, j] *= ratio
    check(sdpa, q, cache, [150], 0.25)


@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 25, 2.0 ** -25, 2.0 ** 40])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 4), (128, 16)])
def test_groups_of_channels_of_unlike_size(sdpa, d, G, ratio):
    import torch
    cache = make(sdpa, 4, 1, 1, 300, d, [300], 9)
    cache[3][..., 1, :] *= ratio
    check(sdpa, rnd((1, G, d), 10), cache, [300], d ** -0.5)
    assert torch.isfinite(cache[3]).all()


@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 25, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("every", [1, 2, 7, 32, 64])
@pytest.mark.parametrize("d,G", [(64, 2), (128, 8)])
def test_values_of_unlike_size_that_count(sdpa, d, G, ratio, every):
    """Large and small rows in turn, by rows and by stretches of rows, all with weight: the large ones set what is exact."""
    cache = make(sdpa, 4, 1, 1, 520, d, [520], 11)
    for j in range(520):
        if (j // every) % 2:
            cache[3][0, 0, j] *= ratio
    check(sdpa, rnd((1, G, d), 12), cache, [520], d ** -0.5)
    flipped = list(cache)
    flipped[3] = cache[3].clone()
    flipped[3][0, 0] = cache[3][0, 0].flip(0)
    check(sdpa, rnd((1, G, d), 12), flipped, [520], d ** -0.5)


def test_rows_of_one_value(sdpa):
    """Groups whose channels are all equal have a scale of 0, some rows, whole stretches or the whole cache."""
    import torch
    d, n = 128, 400
    q = rnd((1, 4, d), 13)
    for rows in (slice(0, 1), slice(3, 200), slice(0, n), slice(390, n)):
        cache = make(sdpa, 4, 1, 1, n, d, [n], 14)
        cache[3][0, 0, rows, :, 0] = 0.0
        check(sdpa, q, cache, [n], d ** -0.5)
        cache[3][0, 0, rows, 1, 0] = 3.0
        check(sdpa, q, cache, [n], d ** -0.5)
    cache = make(sdpa, 4, 1, 1, n, d, [n], 15)
    cache[3][..., 0] = torch.where(rnd((1, 1, n, d // 32), 16).float() > 0, 0.0, 2.0 ** -100)  # and the smallest scales
    cache[3][..., 1] = 0.0
    check(sdpa, q, cache, [n], d ** -0.5)


def test_an_undefined_row_of_values(sdpa):
    """A row whose values are NaN reaches the channels of its groups in the heads that see it, and nothing else."""
    import torch
    d, n = 128, 200
    q, cache = rnd((1, 8, d), 17), make(sdpa, 4, 1, 2, n, d, [n], 18)
    acc, acc2 = (torch.zeros((1, 2, n), device="cuda") for _ in range(2))
    O, L = sdpa.decode_kv4(q, sdpa.Kv4Cache(*cache), i32([n]), acc=acc)
    cache[3][0, 1, 77, 2] = float("nan")
    O2, L2 = sdpa.decode_kv4(q, sdpa.Kv4Cache(*cache), i32([n]), acc=acc2)
    assert torch.isnan(O2[0, 4:, 64:96]).all() and torch.equal(L, L2) and torch.equal(acc, acc2)
    O2[0, 4:, 64:96] = O[0, 4:, 64:96]
    assert torch.equal(O, O2)
