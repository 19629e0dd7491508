"""Prefills and decodes with the largest scales: scale log2 e is beyond 32 bits, a score of 0 still is 0."""
import math

import pytest
from test_cache_gpu import i32, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa(cuda_device):
    import memory_optimal_sdpa_b200 as m
    yield m
    assert m.get_last_device_error() == m.SDPA_OK


@pytest.mark.parametrize("scale", [1e38, 2.5e38, 3.4028234e38, -3.4028234e38])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("call", ["fwd", "fwd_window", "decode", "decode_noalloc", "decode_gqa", "decode_gqa, groups of 4"])
def test_keys_at_and_below_zero(sdpa, call, d, scale):
    """Half of the keys score 0, the others so far below that they weigh nothing."""
    import torch
    n, Hkv = 700, 2
    H = Hkv * (4 if call.endswith("4") else 1)
    q, k = torch.zeros((1, H, d), device="cuda"), torch.zeros((1, Hkv, n, d), device="cuda")
    q[..., 3], q[..., 7] = 200.0, -3.0  # times the scale beyond 32 bits too
    k[:, :, 1::2, 7] = math.copysign(0.5, scale)
    q, k, v = q.to(torch.bfloat16), k.to(torch.bfloat16), rnd((1, Hkv, n, d), 1)
    if call.startswith("fwd"):
        args = (n, 0) if call == "fwd_window" else ()
        O, L = getattr(sdpa, call)(q[:, :, None].contiguous(), k, v, *args, scale=scale)
        O, L = O[:, :, 0], L[:, :, 0]
    else:
        O, L = getattr(sdpa, call.split(",")[0])(q, k, v, i32([n]), scale=scale)
    want = v[:, :, ::2].double().mean(2).repeat_interleave(H // Hkv, 1)
    # 350 equal weights: exact in their sums but for 350 roundings, then O to bf16
    assert ((O.double() - want).abs() <= 2.0 ** -8 * want.abs() + 350 * 2.0 ** -24 * 4).all()
    assert ((L.double() - math.log(n // 2)).abs() <= 1e-5).all()
