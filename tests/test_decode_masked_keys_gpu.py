"""Decodes over a bf16 cache with keys that score -inf: they count nothing, in every place of a split, and where all keys of a
sequence do, O = 0 and LSE = -inf."""
import math

import pytest
from test_cache_gpu import i32, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa(cuda_device):
    import memory_optimal_sdpa_b200 as m
    yield m
    assert m.get_last_device_error() == m.SDPA_OK


@pytest.mark.parametrize("d,G", [(64, 1), (128, 1), (64, 4), (128, 4), (128, 24)])
@pytest.mark.parametrize("call", ["decode", "decode_noalloc", "decode_gqa"])
@pytest.mark.parametrize("lo,hi", [(0, 64), (0, 512), (64, 128), (0, 1100), (500, 1100), (0, 1099), (1, 1100)])
def test_keys_of_minus_infinity(sdpa, lo, hi, call, d, G):
    import torch
    if call != "decode_gqa" and G > 1:
        pytest.skip("one query head for each key/value head")
    n, Hkv = 1100, 2
    q, k, v = rnd((2, Hkv * G, d), 1), rnd((2, Hkv, n, d), 2), rnd((2, Hkv, n, d), 3)
    q[..., 5] = q[..., 5].abs() + 0.5
    run = getattr(sdpa, call)
    hidden = k.clone()
    hidden[0, 1, lo:hi, 5] = -math.inf
    (O, L), (O2, L2) = run(q, hidden, v, i32([n, n])), run(q, k, v, i32([n, n]))
    for b, h in ((0, 0), (1, 0), (1, 1)):
        at = slice(h * G, h * G + G)
        assert torch.equal(O[b, at], O2[b, at]) and torch.equal(L[b, at], L2[b, at])
    at, rest = slice(G, 2 * G), [j for j in range(n) if not lo <= j < hi]
    if not rest:
        assert (O[0, at] == 0).all() and (L[0, at] == -math.inf).all()
        return
    s = q[0, at].double() @ k[0, 1, rest].double().T * d ** -0.5
    want = torch.softmax(s, -1) @ v[0, 1, rest].double()
    # weights and output rounded to bf16, values of order 1
    assert ((O[0, at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * (torch.softmax(s, -1) @ v[0, 1, rest].double().abs())).all()
    assert ((L[0, at].double() - torch.logsumexp(s, -1)).abs() <= 1e-3).all()
