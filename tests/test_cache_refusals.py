"""Calls of the bounded decode cache that have no sound answer are refused, in the binding and in the C ABI (CPU)."""
import pytest

torch = pytest.importorskip("torch")
sdpa = pytest.importorskip("memory_optimal_sdpa_b200")

bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def cache(B=2, H=2, n=8, d=64):
    return sdpa.Kv4Cache(t(B, H, n, d // 2, dtype=u8), t(B, H, n, d // 32, 2), t(B, H, n, d // 2, dtype=u8), t(B, H, n, d // 32, 2))


LENS = t(2, dtype=i32)


def test_no_heads_to_fill_an_output_from():
    """Without a query head there is nothing to launch, so weights, kept rows and new lengths would be left as memory was found."""
    acc, kv = t(2, 2, 8, dtype=f32), t(2, 2, 8, 64)
    for call in (lambda: sdpa.fwd_acc(t(2, 0, 3, 64), kv, t(2, 0, 3, dtype=f32)),
                 lambda: sdpa.fwd_acc(t(2, 0, 3, 64), kv, t(2, 0, 3, dtype=f32), acc, acc_out=acc.clone()),
                 lambda: sdpa.decode_acc(t(2, 0, 64), kv, kv, LENS, acc), lambda: sdpa.decode_kv4(t(2, 0, 64), cache(), LENS, acc_out=acc),
                 lambda: sdpa.evict(t(2, 0, 8, 64), t(2, 0, 8, 64), t(2, 0, 8, dtype=f32), LENS, 4),
                 lambda: sdpa.kv4_evict(cache(H=0), t(2, 0, 8, dtype=f32), LENS, 4)):
        with pytest.raises(ValueError, match="at least one head"):
            call()
