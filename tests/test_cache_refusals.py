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


def test_sums_that_overlap_in_part():
    """acc and acc_out are one array or apart; so are the rows read back, and what an eviction returns."""
    P, FAR, inv = 0x10000, 1 << 40, sdpa.SDPA_ERR_INVALID_ARG
    lib, size = sdpa.lib, 2 * 8 * 4  # two heads, eight rows
    for out in (P + 4, P + size - 4, P - 4):
        assert lib.sdpa_decode_acc(FAR, FAR, FAR, FAR, FAR, None, P, out, 1, 2, 2, 8, 64, 0.1, FAR, 1 << 30, None) == inv
        assert lib.sdpa_decode_kv4(FAR, FAR, FAR, FAR, FAR, FAR, FAR, None, P, out, 1, 2, 2, 8, 64, 0.1, FAR, 1 << 30, None) == inv
        assert lib.sdpa_fwd_acc(FAR, FAR, FAR, P, out, 1, 2, 2, 4, 8, 8, 64, 0.1, 0, None) == inv
    # apart, or one: the arguments are right (what is refused next is the missing workspace, or the device here)
    for out in (P, P + size, P - size):
        assert lib.sdpa_decode_acc(FAR, FAR, FAR, FAR, FAR, None, P, out, 1, 2, 2, 8, 64, 0.1, None, 0, None) == sdpa.SDPA_ERR_WORKSPACE
    rows = 2 * 3 * 64 * 2
    for read in (P + 16, P + rows - 16):
        assert lib.sdpa_kv4_append(FAR, 2 * FAR, FAR, None, FAR, FAR, FAR, FAR, P, read, 1, 2, 3, 8, 64, None) == inv

    def evict(keep, new, lens=3 * FAR):
        return lib.sdpa_evict(FAR, 2 * FAR, 4 * FAR, lens, FAR, 2 * FAR, 4 * FAR, keep, new, 1, 2, 8, 8, 64, 4, 1, None)
    assert evict(FAR + 64, 5 * FAR) == inv and evict(4 * FAR, 5 * FAR) == inv and evict(3 * FAR, 5 * FAR) == inv
    assert evict(5 * FAR, 5 * FAR + 4) == inv and evict(5 * FAR, 2 * FAR) == inv
