"""The bounded decode cache on the GPU, against plain 64-bit computations of its definitions.

Rounding: a result rounded to bf16 is off by at most 2^-8 of its value.  A score is a sum of d products of
|q| |k| held in 32 bits: with the accumulation of the tensor cores counted as one unit (2^-23) per addition it
is off by at most (d + 16) 2^-23 |q|_2 |k|_2 |scale| =: delta, and a weight exp(score - LSE) by a factor
1 +- (4 delta + 2^-18) (the score, the LSE, two exponentials; 2^-18 for weights used as two bf16 parts).
"""
import math
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def sdpa(cuda_device):
    import memory_optimal_sdpa_b200 as m
    yield m
    assert m.get_last_device_error() == m.SDPA_OK


def rnd(shape, seed, std=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def i32(values):
    import torch
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def nan_rows(t, lens):
    """NaN (all bits set for bytes) in the rows at and past each sequence's length."""
    for b, n in enumerate(lens):
        t[b, :, n:] = 255 if t.dtype.itemsize == 1 else float("nan")
    return t


def code_index(d):
    """Byte and shift of each channel's code, from the layout's description."""
    ng = d // 32
    ch = np.arange(d)
    g, r, e = ch // 32, ch % 32 // 4, ch % 4 // 2
    return 2 * (r * ng + g) + e, 4 * (ch % 2)


def values64(codes, scales):
    """What a 4-bit cache stands for, in 64 bits."""
    import torch
    d = codes.shape[-1] * 2
    byte, shift = code_index(d)
    byte, shift = torch.from_numpy(byte).to(codes.device), torch.from_numpy(shift).to(codes.device)
    c = (codes[..., byte].int() >> shift) & 15
    s = scales.double().repeat_interleave(32, dim=-2)
    return s[..., 0] * c + s[..., 1]


def random_cache(sdpa, B, H, cap, d, lens, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    c = []
    for _ in "kv":
        codes = (rand(B, H, cap, d // 2) * 256).to(torch.uint8)
        s = 0.1 + 0.3 * rand(B, H, cap, d // 32)
        m = -s * 15 * rand(B, H, cap, d // 32) + rand(1, H, 1, d // 32) - 0.5
        c += [nan_rows(codes, lens), nan_rows(torch.stack((s, m), -1).to(torch.bfloat16), lens)]
    return sdpa.Kv4Cache(*c)


# ------------------------------------------------------------------------------------------ append and load
def bf16_up(x):
    """The smallest non-negative bf16 number not below the Fraction x >= 0, by bisection over its bits."""
    def value(bits):
        e, f = bits >> 7, bits & 127
        return Fraction(f, 128) * Fraction(2) ** -126 if e == 0 else (1 + Fraction(f, 128)) * Fraction(2) ** (e - 127)
    lo, hi = 0, 0x7F7F
    while lo < hi:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if value(mid) >= x else (mid + 1, hi)
    return value(lo)


def quantise_exact(group):
    """(codes, scale, minimum) of 32 finite numbers, in rational arithmetic."""
    x = [Fraction(float(v)) for v in group]
    m = min(x)
    s = bf16_up((max(x) - m) / 15)
    return [round((v - m) / s) if s else 0 for v in x], s, m  # round(): halves to even


def check_groups(rows, codes, scales, read):
    """Every group of bf16 rows [N, d] against the rational definition."""
    import torch
    d = rows.shape[-1]
    byte, shift = code_index(d)
    x, c = rows.double().cpu().numpy(), codes.cpu().numpy()
    c = (c[:, byte] >> shift) & 15
    sc = scales.double().cpu().numpy()
    rd = read.double().cpu().numpy()
    for n in range(x.shape[0]):
        for g in range(d // 32):
            at = slice(32 * g, 32 * g + 32)
            if not np.isfinite(x[n, at]).all():
                assert np.isnan(sc[n, g]).all() and (c[n, at] == 0).all() and np.isnan(rd[n, at]).all()
                continue
            want, s, m = quantise_exact(x[n, at])
            assert Fraction(float(sc[n, g, 0])) == s and Fraction(float(sc[n, g, 1])) == m
            assert c[n, at].tolist() == want
            value = torch.tensor([float(s * k + m) for k in want], dtype=torch.float32).to(torch.bfloat16)
            assert (value.double().numpy() == rd[n, at]).all()
            assert all(abs(Fraction(float(v)) - (s * k + m)) <= s / 2 for v, k in zip(x[n, at], want))


@pytest.mark.parametrize("d", [64, 128])
def test_append_codes_are_exact(sdpa, d):
    """Groups where rounding can go wrong: ties, constants, offsets, tiny and huge numbers, NaN, infinities."""
    import torch
    rng = np.random.RandomState(d)
    rows = []
    for k in range(48):
        x = rng.randn(d).astype(np.float64)
        x = {0: x, 1: np.round(x * 4), 2: np.full(d, 1.7), 3: 100 + x, 4: x * 1e38, 5: x * 1e-39, 6: x * 1e-20,
             7: np.zeros(d), 8: np.where(rng.rand(d) < 0.5, 3e38, -3e38), 9: x * np.exp(rng.randn(d) * 8),
             10: np.arange(d) % 31 / 2.0, 11: np.arange(d) % 31 * 1e-40}[k % 12]
        rows.append(x)
    x = torch.tensor(np.array(rows), device="cuda").to(torch.bfloat16).clamp(-3.38e38, 3.38e38)
    x[5, 3], x[17, 40], x[29, d - 1] = float("nan"), float("inf"), -float("inf")
    k = x.view(1, 2, 24, d).contiguous()
    v = k.flip(2).contiguous()
    c = sdpa.kv4_cache(1, 2, 30, d)
    kr, vr = torch.zeros_like(k), torch.zeros_like(v)
    sdpa.kv4_append(c, k, v, i32([6]), k_read=kr, v_read=vr)
    for rows, codes, scales, read in ((k, c.k_codes, c.k_scales, kr), (v, c.v_codes, c.v_scales, vr)):
        assert (codes[:, :, :6] == 0).all() and (scales[:, :, :6] == 0).all()
        check_groups(rows.view(-1, d), codes[:, :, 6:].reshape(48, -1), scales[:, :, 6:].reshape(48, -1, 2), read.view(-1, d))


@pytest.mark.parametrize("B,H,n,d,lens,n_new,cap", [
    (1, 1, 1, 64, [0], None, 1), (1, 1, 1, 128, [4], None, 5), (3, 5, 1, 128, [0, 7, 30], None, 31),
    (2, 3, 37, 64, [0, 11], [37, 0], 48), (4, 1, 130, 128, [1, 0, 3, 9], [129, 130, 1, 64], 140),
    (2, 7, 1001, 64, [5, 0], [1000, 3], 1005)])
def test_append_and_load(sdpa, B, H, n, d, lens, n_new, cap):
    import torch
    k, v = rnd((B, H, n, d), 1), rnd((B, H, n, d), 2, 3.0)
    c = sdpa.Kv4Cache(*(torch.full_like(t, 7) for t in sdpa.kv4_cache(B, H, cap, d)))
    kr, vr = torch.full_like(k, 5), torch.full_like(v, 5)
    sdpa.kv4_append(c, k, v, i32(lens), n_new=None if n_new is None else i32(n_new), k_read=kr, v_read=vr)
    new = n_new or [n] * B
    ends = [a + m for a, m in zip(lens, new)]
    K, V = (torch.full((B, H, cap + 3, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert sdpa.kv4_load(c, i32(ends), k=K, v=V)[0] is K
    for rows, codes, scales, read, out in ((k, c.k_codes, c.k_scales, kr, K), (v, c.v_codes, c.v_scales, vr, V)):
        want = values64(codes, scales)
        for b in range(B):
            at = slice(lens[b], ends[b])
            assert (codes[b, :, :lens[b]] == 7).all() and (codes[b, :, ends[b]:] == 7).all()
            assert (scales[b, :, :lens[b]] == 7).all() and (scales[b, :, ends[b]:] == 7).all()
            assert (read[b, :, new[b]:] == 5).all() and (out[b, :, ends[b]:] == 9).all()
            step = scales[b, :, at, :, 0].double().repeat_interleave(32, dim=-1)
            assert ((rows[b, :, :new[b]].double() - want[b, :, at]).abs() <= step / 2).all()
            assert torch.equal(read[b, :, :new[b]], out[b, :, at])
            assert torch.equal(out[b, :, :ends[b]], want[b, :, :ends[b]].float().to(torch.bfloat16))
    # fewer rows than cached, and tensors made by the call
    short = max(1, cap // 2)
    K2, V2 = sdpa.kv4_load(c, i32(ends), n_rows=short)
    for b in range(B):
        m = min(short, ends[b])
        assert torch.equal(K2[b, :, :m], K[b, :, :m]) and (K2[b, :, m:] == 0).all() and torch.equal(V2[b, :, :m], V[b, :, :m])


def test_bad_lengths_are_reported(sdpa):
    import torch
    d, cap = 64, 8
    c = sdpa.kv4_cache(2, 1, cap, d)
    rows = rnd((2, 1, 4, d), 3)
    bad = sdpa.SDPA_ERR_DEVICE_BAD_LENGTH
    guard = [t.clone() for t in c]
    for lens, n_new in (([6, 0], None), ([-1, 0], None), ([9, 0], None), ([0, 0], [5, 1]), ([0, 0], [-1, 1])):
        sdpa.kv4_append(c, rows, rows, i32(lens), n_new=None if n_new is None else i32(n_new))
        assert sdpa.get_last_device_error() == bad
    q, acc = rnd((2, 2, d), 4), torch.zeros((2, 1, cap), device="cuda")
    kv, kv2 = rnd((2, 1, cap, d), 5), rnd((2, 1, cap, d), 6)
    for lens in ([9, 1], [-1, 1]):
        for call in (lambda: sdpa.decode_kv4(q, c, i32(lens), acc=acc), lambda: sdpa.kv4_load(c, i32(lens)),
                     lambda: sdpa.decode_acc(q, kv, kv, i32(lens), acc), lambda: sdpa.evict(kv, kv2, acc, i32(lens), 3),
                     lambda: sdpa.kv4_evict(c, acc, i32(lens), 3)):
            call()
            assert sdpa.get_last_device_error() == bad
    assert len(guard) == 4 and sdpa.get_last_device_error() == sdpa.SDPA_OK


# ------------------------------------------------------------------------------------------ decode
def attend64(q, k, v, lens, scale):
    """O, LSE and the group-summed weights in 64 bits from 64-bit keys and values."""
    import torch
    B, Hkv, cap, d = k.shape
    G = q.shape[1] // Hkv
    O = torch.zeros((B, Hkv, G, d), dtype=torch.float64, device="cuda")
    L = torch.full((B, Hkv, G), -math.inf, dtype=torch.float64, device="cuda")
    W = torch.zeros((B, Hkv, cap), dtype=torch.float64, device="cuda")
    delta, vmax = 0.0, 0.0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        qq, kk, vv = q[b].double().view(Hkv, G, d), k[b, :, :n], v[b, :, :n]
        s = torch.einsum("hgd,hnd->hgn", qq, kk) * scale
        L[b] = torch.logsumexp(s, -1)
        p = torch.softmax(s, -1)
        O[b], W[b, :, :n] = torch.einsum("hgn,hnd->hgd", p, vv), p.sum(1)
        delta = max(delta, (d + 16) * 2.0 ** -23 * qq.norm(dim=-1).max().item() * kk.norm(dim=-1).max().item() * abs(scale))
        vmax = max(vmax, vv.abs().max().item())
    return O.view(B, -1, d), L.view(B, -1), W, delta, vmax


def check_decode(O, L, ref, acc_in, acc_out, lens, untouched):
    import torch
    O64, L64, W, delta, vmax = ref
    rel = 4 * delta + 2.0 ** -18
    err = (O.double() - O64).abs()
    assert (err <= HALF_BF16 * O64.abs() + 2 * rel * vmax + 1e-37).all(), err.max().item()
    empty = torch.isinf(L64)
    assert torch.equal(L[empty].double(), L64[empty]) and (O.double()[empty] == 0).all()
    err = (L.double() - L64)[~empty].abs()
    assert (err <= 2 * delta + 2.0 ** -20 * (1 + L64[~empty].abs())).all()
    if acc_out is None:
        return
    heads = O.shape[1] // W.shape[1]
    for b, n in enumerate(lens):
        want = W[b, :, :n] + (0 if acc_in is None else acc_in[b, :, :n].double())
        err = (acc_out[b, :, :n].double() - want).abs()
        # a weight below 2^-126 is not a normal 32-bit number: each of the group's may be off by as much
        assert (err <= rel * W[b, :, :n] + 2.0 ** -22 * want + heads * 2.0 ** -126).all(), err.max().item()
        assert torch.equal(acc_out[b, :, n:], untouched[b, :, n:])


DECODE = [  # B, Hq, Hkv, cap, d, lens
    (1, 1, 1, 1, 64, [1]), (1, 1, 1, 1, 128, [1]), (2, 2, 1, 2, 128, [0, 2]), (3, 8, 8, 70, 64, [0, 1, 70]),
    (2, 8, 1, 257, 128, [255, 257]), (2, 24, 8, 1001, 128, [1000, 33]), (1, 9, 1, 300, 64, [299]), (1, 16, 1, 513, 128, [512]),
    (2, 40, 2, 129, 128, [128, 65]), (1, 17, 1, 31, 64, [31]), (1, 96, 3, 2049, 64, [2047]), (5, 32, 4, 63, 128, [63, 1, 17, 16, 15]),
    (1, 4, 4, 9001, 128, [8999]), (1, 32, 4, 33333, 64, [33333]), (2, 64, 8, 4099, 128, [4099, 1025]),
]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("B,Hq,Hkv,cap,d,lens", DECODE)
def test_decode(sdpa, B, Hq, Hkv, cap, d, lens, bits):
    import torch
    seed = cap + Hq
    q = rnd((B, Hq, d), seed, 1.5)
    scale = d ** -0.5
    if bits == 4:
        c = random_cache(sdpa, B, Hkv, cap, d, lens, seed)
        k64, v64 = values64(c.k_codes, c.k_scales), values64(c.v_codes, c.v_scales)
    else:
        k, v = (nan_rows(rnd((B, Hkv, cap, d), seed + s), lens) for s in (1, 2))
        k64, v64 = k.double(), v.double()
    ref = attend64(q, k64, v64, lens, scale)
    acc = rnd((B, Hkv, cap), seed + 3).float().abs()
    out = torch.full_like(acc, 3.0)
    call = (lambda **kw: sdpa.decode_kv4(q, c, i32(lens), **kw)) if bits == 4 else (lambda **kw: sdpa.decode_acc(q, k, v, i32(lens), **kw))
    O, L = call(acc=acc, acc_out=out)
    check_decode(O, L, ref, acc, out, lens, torch.full_like(acc, 3.0))
    fresh = torch.full_like(acc, 4.0)
    O2, L2 = call(acc_out=fresh)  # from zero
    check_decode(O2, L2, ref, None, fresh, lens, torch.full_like(acc, 4.0))
    inplace = acc.clone()
    O3, L3 = call(acc=inplace)
    assert torch.equal(inplace[:, :, :], torch.where(torch.arange(cap, device="cuda") < i32(lens)[:, None, None], out, acc))
    assert torch.equal(O, O2) and torch.equal(O, O3) and torch.equal(L, L3)
    if bits == 4:
        O4, L4 = call()
        check_decode(O4, L4, ref, None, None, lens, None)
        assert call(want_lse=False)[1] is None


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("bits", [4, 16])
def test_decode_scales(sdpa, bits, scale):
    """Any finite scale; with 2.0 nearly all weight sits on one key."""
    B, Hq, Hkv, cap, d, lens = 2, 12, 3, 300, 64, [300, 131]
    q = rnd((B, Hq, d), 1)
    acc = rnd((B, Hkv, cap), 2).float() * 0
    if bits == 4:
        c = random_cache(sdpa, B, Hkv, cap, d, lens, 3)
        k64, v64 = values64(c.k_codes, c.k_scales), values64(c.v_codes, c.v_scales)
        O, L = sdpa.decode_kv4(q, c, i32(lens), scale=scale, acc=acc)
    else:
        k, v = rnd((B, Hkv, cap, d), 4), rnd((B, Hkv, cap, d), 5)
        k64, v64 = k.double(), v.double()
        O, L = sdpa.decode_acc(q, k, v, i32(lens), acc, scale=scale)
    check_decode(O, L, attend64(q, k64, v64, lens, scale), None, acc, lens, acc * 0)


def test_decode_nan_stays_in_its_head(sdpa):
    """A NaN in one query head reaches that head's output and its group's weights, and nothing else."""
    import torch
    B, Hq, Hkv, cap, d, lens = 1, 4, 2, 200, 128, [150]
    q = rnd((B, Hq, d), 1)
    c = random_cache(sdpa, B, Hkv, cap, d, lens, 2)
    acc = torch.zeros((B, Hkv, cap), device="cuda")
    O, L = sdpa.decode_kv4(q, c, i32(lens), acc=acc)
    q2, acc2 = q.clone(), torch.zeros_like(acc)
    q2[0, 1, 5] = float("nan")
    O2, L2 = sdpa.decode_kv4(q2, c, i32(lens), acc=acc2)
    assert torch.isnan(O2[0, 1]).all() and torch.isnan(L2[0, 1]) and torch.isnan(acc2[0, 0, :150]).all()
    rest = [0, 2, 3]
    assert torch.equal(O[0, rest], O2[0, rest]) and torch.equal(L[0, rest], L2[0, rest]) and torch.equal(acc[0, 1], acc2[0, 1])
    assert (acc2[0, 0, 150:] == 0).all()


# ------------------------------------------------------------------------------------------ weights of a prompt
PROMPT = [  # B, Hq, Hkv, n_q, n_kv, d, causal
    (1, 1, 1, 1, 1, 64, False), (1, 1, 1, 1, 1, 128, True), (2, 3, 1, 1, 129, 128, True), (1, 2, 2, 128, 128, 64, True),
    (1, 4, 2, 127, 255, 128, True), (2, 2, 1, 300, 100, 64, True), (1, 6, 2, 65, 1000, 128, False), (1, 5, 1, 257, 257, 128, True),
    (3, 2, 2, 64, 513, 64, True), (1, 8, 2, 1024, 1024, 128, True), (1, 2, 1, 700, 640, 64, False), (1, 1, 1, 129, 2, 128, True),
    # several units per block with one, two, an odd and many query tiles each, for narrow and wide units
    (4, 8, 8, 100, 1100, 64, True), (4, 8, 8, 200, 1000, 128, False), (2, 24, 8, 380, 1500, 64, True), (2, 6, 2, 1300, 6000, 128, True),
    (2, 16, 8, 520, 2500, 64, True), (2, 16, 8, 600, 2600, 128, False), (4, 20, 4, 300, 2400, 128, True),
]


@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,d,causal", PROMPT)
def test_fwd_acc(sdpa, B, Hq, Hkv, n_q, n_kv, d, causal):
    import torch
    q, k = rnd((B, Hq, n_q, d), 1), rnd((B, Hkv, n_kv, d), 2)
    scale = d ** -0.5
    G = Hq // Hkv
    s = torch.einsum("bhgid,bhjd->bhgij", q.double().view(B, Hkv, G, n_q, d), k.double()) * scale
    if causal:
        s.masked_fill_(torch.arange(n_kv, device="cuda") > torch.arange(n_q, device="cuda")[:, None] + (n_kv - n_q), -math.inf)
    lse64 = torch.logsumexp(s, -1)
    lse = lse64.float().view(B, Hq, n_q)  # -inf for the queries that see no key
    w = torch.exp(s - torch.where(torch.isinf(lse64), torch.zeros_like(lse64), lse.view_as(lse64).double())[..., None]).sum((2, 3))
    delta = (d + 16) * 2.0 ** -23 * q.double().norm(dim=-1).max().item() * k.double().norm(dim=-1).max().item() * scale
    rel = 2 * delta + 2.0 ** -18 + 2.0 ** -22 * math.sqrt(n_q * G)
    tiny = n_q * G * 2.0 ** -126  # weights below 2^-126 are not normal 32-bit numbers
    acc = rnd((B, Hkv, n_kv + 5), 3).float().abs()
    out = torch.full_like(acc, 3.0)
    assert sdpa.fwd_acc(q, k, lse, acc, causal=causal, acc_out=out) is out
    want = acc[:, :, :n_kv].double() + w
    assert ((out[:, :, :n_kv].double() - want).abs() <= rel * w + 2.0 ** -23 * want + tiny).all()
    assert (out[:, :, n_kv:] == 3).all()
    fresh = sdpa.fwd_acc(q, k, lse, causal=causal)
    assert fresh.shape == (B, Hkv, n_kv) and ((fresh.double() - w).abs() <= rel * w + tiny).all()
    before = acc.clone()
    assert sdpa.fwd_acc(q, k, lse, acc, causal=causal) is acc
    assert torch.equal(acc[:, :, :n_kv], out[:, :, :n_kv]) and torch.equal(acc[:, :, n_kv:], before[:, :, n_kv:])


@pytest.mark.parametrize("scale", [0.0, -0.25, 1.0])
def test_fwd_acc_with_fwd(sdpa, scale):
    """With the LSE that the prefill wrote: every query that sees a key hands out a weight of one."""
    import torch
    B, H, n_q, n_kv, d = 2, 3, 330, 290, 128
    q, k, v = rnd((B, H, n_q, d), 1), rnd((B, H, n_kv, d), 2), rnd((B, H, n_kv, d), 3)
    _, lse = sdpa.fwd(q, k, v, causal=True, scale=scale)
    acc = sdpa.fwd_acc(q, k, lse, causal=True, scale=scale)
    seen = n_q - max(0, n_q - n_kv)
    # the prefill's LSE is off by at most 1e-3
    assert ((acc.double().sum(-1) - seen).abs() <= 2e-3 * seen).all()


def test_fwd_acc_nan_stays_in_its_group(sdpa):
    """A NaN in one query reaches the weights of every key that its group's query sees, and nothing else; an infinite
    LSE takes a query out."""
    import torch
    B, Hq, Hkv, n, d = 1, 4, 2, 256, 64
    q, k, v = rnd((B, Hq, n, d), 1), rnd((B, Hkv, n, d), 2), rnd((B, Hkv, n, d), 3)
    _, lse = sdpa.fwd(q, k.repeat_interleave(2, 1).contiguous(), v.repeat_interleave(2, 1).contiguous(), causal=True)
    acc = sdpa.fwd_acc(q, k, lse, causal=True)
    for row in (*range(96, 104), *range(160, 168), 255):
        q2 = q.clone()
        q2[0, 1, row, 7] = float("nan")
        bad = sdpa.fwd_acc(q2, k, lse, causal=True)
        assert torch.isnan(bad[0, 0, :row + 1]).all() and torch.equal(bad[0, 0, row + 1:], acc[0, 0, row + 1:])
        assert torch.equal(bad[0, 1], acc[0, 1])
    l2 = lse.clone()
    l2[0, :, :200] = float("inf")
    l2[0, :, 77] = -float("inf")
    few = sdpa.fwd_acc(q, k, l2, causal=True)
    last = sdpa.fwd_acc(q[:, :, 200:].contiguous(), k, lse[:, :, 200:].contiguous(), causal=True)
    # the same weights, summed in another order: 56 queries of two heads
    assert ((few - last).abs() <= 112 * 2.0 ** -23 * last).all()


@pytest.mark.parametrize("n_q", [1, 40, 64, 129])
@pytest.mark.parametrize("causal", [False, True])
def test_fwd_acc_key_of_minus_infinity(sdpa, n_q, causal):
    """A key whose scores are all -inf weighs 0 and changes nothing else, for any number of queries."""
    import torch
    n_kv, d = 200, 64
    q, k = rnd((1, 4, n_q, d), 1), rnd((1, 2, n_kv, d), 2)
    q[..., 5] = q[..., 5].abs() + 0.5
    s = torch.einsum("bhgid,bhjd->bhgij", q.double().view(1, 2, 2, n_q, d), k.double()) / 8
    s[..., 30] = -math.inf
    if causal:
        s.masked_fill_(torch.arange(n_kv, device="cuda") > torch.arange(n_q, device="cuda")[:, None] + (n_kv - n_q), -math.inf)
    lse = torch.logsumexp(s, -1).float().view(1, 4, n_q)
    plain = sdpa.fwd_acc(q, k, lse, causal=causal)
    k[:, :, 30, 5] = -math.inf
    acc = sdpa.fwd_acc(q, k, lse, causal=causal)
    assert (acc[..., 30] == 0).all()
    acc[..., 30] = plain[..., 30]
    assert torch.equal(acc, plain)


def test_fwd_acc_without_queries(sdpa):
    import torch
    k = rnd((1, 2, 7, 64), 1)
    acc = rnd((1, 2, 9), 2).float()
    out = torch.full_like(acc, 3.0)
    q, lse = torch.empty((1, 4, 0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 4, 0), device="cuda")
    sdpa.fwd_acc(q, k, lse, acc, acc_out=out)
    assert torch.equal(out[:, :, :7], acc[:, :, :7]) and (out[:, :, 7:] == 3).all()
    assert (sdpa.fwd_acc(q, k, lse) == 0).all()


# ------------------------------------------------------------------------------------------ eviction
def kept_rows(acc, n, budget, recent):
    """The rows kept of one sequence and head, by the definition (NaN lowest, the lower row where equal)."""
    new = min(n, budget)
    rec = min(recent, new)
    w = [-math.inf if math.isnan(x) else x for x in acc[:n - rec].tolist()]
    nan = [math.isnan(x) for x in acc[:n - rec].tolist()]
    best = sorted(range(n - rec), key=lambda j: (nan[j], -w[j], j))[:new - rec]
    return sorted(best) + list(range(n - rec, n))


def weights_for(kind, shape, seed):
    import torch
    w = rnd(shape, seed).float().exp()
    if kind == "ties":
        w = (w * 2).round() / 2
    elif kind == "special":
        pick = rnd(shape, seed + 1).float()
        w = torch.where(pick > 1.2, math.nan, torch.where(pick > 0.8, math.inf, torch.where(pick > 0.4, -0.0, torch.where(pick > 0, 0.0, torch.where(pick < -1, -math.inf, -w)))))
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    return w


EVICT = [  # B, H, cap, out cap (None: in place), d, lens, budget, recent
    (1, 1, 1, None, 64, [1], 1, 0), (1, 2, 8, None, 128, [8], 1, 1), (3, 2, 40, None, 64, [0, 40, 17], 20, 5),
    (2, 3, 700, 300, 128, [700, 299], 300, 0), (2, 2, 1500, None, 64, [1499, 1024], 1023, 64), (1, 2, 5000, 77, 128, [4999], 77, 77),
    (1, 1, 20001, None, 64, [20001], 10000, 600), (2, 1, 33, 40, 64, [33, 1], 40, 3), (1, 3, 40000, 4096, 64, [39999], 4000, 100),
]


@pytest.mark.parametrize("kind", ["plain", "ties", "special", "equal"])
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("B,H,cap,n_out,d,lens,budget,recent", EVICT)
def test_evict(sdpa, B, H, cap, n_out, d, lens, budget, recent, bits, kind):
    import torch
    acc = nan_rows(weights_for(kind, (B, H, cap), 7), lens)
    if bits == 4:
        arrays = list(random_cache(sdpa, B, H, cap, d, lens, 8))
    else:
        arrays = [nan_rows(rnd((B, H, cap, d), s), lens) for s in (1, 2)]
    before, acc_before = [a.clone() for a in arrays], acc.clone()
    if n_out is None:
        outs, acc_out, kw = arrays, acc, {}
    else:
        outs = [torch.full((B, H, n_out, *a.shape[3:]), 3, dtype=a.dtype, device="cuda") for a in arrays]
        acc_out = torch.full((B, H, n_out), 3.0, device="cuda")
        kw = dict(out=sdpa.Kv4Cache(*outs), acc_out=acc_out) if bits == 4 else dict(k_out=outs[0], v_out=outs[1], acc_out=acc_out)
    tail = [o.clone() for o in outs]
    lens_d = i32(lens)
    if bits == 4:
        keep, new = sdpa.kv4_evict(sdpa.Kv4Cache(*arrays), acc, lens_d, budget, recent=recent, **kw)
    else:
        keep, new = sdpa.evict(*arrays, acc, lens_d, budget, recent=recent, **kw)
    assert new.tolist() == [min(n, budget) for n in lens] and lens_d.tolist() == lens
    bits_of = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    for b, n in enumerate(lens):
        for h in range(H):
            rows = kept_rows(acc_before[b, h].cpu(), n, budget, recent)
            m = len(rows)
            assert keep[b, h].tolist() == rows + [-1] * (budget - m)
            assert torch.equal(bits_of(acc_out[b, h, :m]), bits_of(acc_before[b, h, rows])) and (acc_out[b, h, m:] == 0).all()
            for o, src, old in zip(outs, before, tail):
                assert torch.equal(bits_of(o[b, h, :m]), bits_of(src[b, h, rows]))
                assert torch.equal(bits_of(o[b, h, m:]), bits_of(old[b, h, m:]))
    if n_out is not None:  # the inputs stay
        assert all(torch.equal(bits_of(a), bits_of(x)) for a, x in zip(arrays, before)) and torch.equal(bits_of(acc), bits_of(acc_before))


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("d,G", [(128, 4), (64, 1)])
def test_serving_run(sdpa, d, G):
    """A prompt, its weights, eviction, the 4-bit cache, decode steps that append and keep the weights, a second
    eviction, and the rows back as bf16 for the next turn: each step against 64 bits on what the step before gave."""
    import torch
    B, Hkv, n, cap, budget = 2, 2, 400, 160, 150
    H, scale = Hkv * G, d ** -0.5
    q, k, v = rnd((B, H, n, d), 1), rnd((B, Hkv, n, d), 2), rnd((B, Hkv, n, d), 3)
    wide = lambda t: t.repeat_interleave(G, dim=1).contiguous()  # noqa: E731
    _, lse = sdpa.fwd(q, wide(k), wide(v), causal=True)
    acc = sdpa.fwd_acc(q, k, lse, causal=True)
    assert ((acc.sum(-1) - n * G).abs() <= 2e-3 * n * G).all()
    k1, v1 = (torch.zeros((B, Hkv, cap, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    acc1 = torch.zeros((B, Hkv, cap), device="cuda")
    keep, lens = sdpa.evict(k, v, acc, i32([n, n]), budget, recent=32, k_out=k1, v_out=v1, acc_out=acc1)
    for b in range(B):
        for h in range(Hkv):
            assert keep[b, h].tolist() == kept_rows(acc[b, h].cpu(), n, budget, 32)
    cache = sdpa.kv4_cache(B, Hkv, cap, d)
    sdpa.kv4_append(cache, k1, v1, i32([0, 0]), n_new=lens)
    for step in range(30):
        kn, vn, qn = (rnd((B, h, 1, d), 100 + 3 * step + i) for i, h in enumerate((Hkv, Hkv, H)))
        if lens[0].item() == cap:
            before = acc1.clone()
            keep, lens = sdpa.kv4_evict(cache, acc1, lens, budget, recent=32)
            assert lens.tolist() == [budget] * B and keep[1, 1].tolist() == kept_rows(before[1, 1].cpu(), cap, budget, 32)
        sdpa.kv4_append(cache, kn, vn, lens)
        lens = lens + 1
        before = acc1.clone()
        O, L = sdpa.decode_kv4(qn.view(B, H, d), cache, lens, acc=acc1)
        ref = attend64(qn.view(B, H, d), values64(cache.k_codes, cache.k_scales), values64(cache.v_codes, cache.v_scales), lens.tolist(), scale)
        check_decode(O, L, ref, before, acc1, lens.tolist(), before)
    m = int(lens[0])
    kb, vb = sdpa.kv4_load(cache, lens, n_rows=m)
    q2 = rnd((B, H, 5, d), 999)
    O, _ = sdpa.fwd(q2, wide(kb), wide(vb), causal=False)
    s = torch.einsum("bhid,bhjd->bhij", q2.double(), wide(kb).double()) * scale
    ref = torch.einsum("bhij,bhjd->bhid", torch.softmax(s, -1), wide(vb).double())
    # the prefill's tolerance: weights and output rounded to bf16
    assert ((O.double() - ref).abs() <= 1e-2 + 1e-2 * ref.abs()).all()


def test_given_outputs_workspace_and_stream(sdpa):
    """Outputs, workspaces and a stream from the caller give what the plain calls give; a workspace too small is refused."""
    import torch
    B, Hq, Hkv, cap, d, lens = 2, 12, 4, 500, 128, [500, 77]
    q, kv, vv = rnd((B, Hq, d), 1), rnd((B, Hkv, cap, d), 2), rnd((B, Hkv, cap, d), 3)
    c = random_cache(sdpa, B, Hkv, cap, d, lens, 4)
    acc = rnd((B, Hkv, cap), 5).float()
    n = i32(lens)
    side = torch.cuda.Stream()
    for call, size in ((lambda **kw: sdpa.decode_kv4(q, c, n, acc=acc, **kw), sdpa.decode_kv4_workspace_size(B, Hq, Hkv, cap, d, True)),
                       (lambda **kw: sdpa.decode_acc(q, kv, vv, n, acc, **kw), sdpa.decode_acc_workspace_size(B, Hq, Hkv, cap, d))):
        out = torch.zeros_like(acc)
        O, L = call(acc_out=out)
        o, lse, ws = torch.empty_like(q), torch.empty((B, Hq), device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
        out2 = torch.zeros_like(acc)
        torch.cuda.synchronize()
        O2, L2 = call(o=o, lse=lse, workspace=ws, acc_out=out2, stream=side)
        side.synchronize()
        assert O2 is o and L2 is lse and torch.equal(O, O2) and torch.equal(L, L2) and torch.equal(out, out2)
        out3 = torch.zeros_like(acc)
        torch.cuda.synchronize()
        O3, L3 = call(acc_out=out3, stream=side)
        side.synchronize()
        assert torch.equal(O, O3) and torch.equal(L, L3) and torch.equal(out, out3)
        with pytest.raises(sdpa.SdpaError, match="WORKSPACE"):
            call(acc_out=out, workspace=ws[:-16])
    torch.cuda.synchronize()
    k, v = sdpa.kv4_load(c, n, stream=side)
    side.synchronize()
    assert torch.equal(k, sdpa.kv4_load(c, n)[0])
    w = sdpa.fwd_acc(q[:, :, None].contiguous(), kv, L[:, :, None].contiguous(), stream=side)
    keep, new = sdpa.kv4_evict(c, acc.clone(), n, 60, recent=7, stream=side)
    side.synchronize()
    assert w.shape == (B, Hkv, cap) and new.tolist() == [60, 60] and keep[1, 0, -7:].tolist() == list(range(70, 77))


def test_streams_and_graphs(sdpa):
    """A decode step captured once and replayed as the cache grows, beside eager calls on another stream."""
    import torch
    B, Hq, Hkv, cap, d = 2, 8, 2, 96, 64
    q, kn, vn = rnd((B, Hq, d), 1), rnd((B, Hkv, 1, d), 2), rnd((B, Hkv, 1, d), 3)
    def fresh():
        c = sdpa.kv4_cache(B, Hkv, cap, d)
        sdpa.kv4_append(c, rnd((B, Hkv, 60, d), 4), rnd((B, Hkv, 60, d), 5), i32([0, 0]))
        return c, torch.zeros((B, Hkv, cap), device="cuda"), i32([60, 41])
    def step(c, acc, lens):
        sdpa.kv4_append(c, kn, vn, lens)
        lens += 1
        return sdpa.decode_kv4(q, c, lens, acc=acc)
    want = fresh()
    for _ in range(5):
        O, L = step(*want)
    side = torch.cuda.Stream()
    got = fresh()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(*got)  # on the side stream, eagerly
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O2, L2 = step(*got)
    two = fresh()
    with torch.cuda.graph(other):
        O3, L3 = step(*two)
    for _ in range(4):
        graph.replay()
        other.replay()
    torch.cuda.synchronize()
    assert got[2].tolist() == [65, 46] and torch.equal(O, O2) and torch.equal(L, L2)
    assert torch.equal(got[1], want[1]) and all(torch.equal(a, b) for a, b in zip(got[0], want[0]))
    other.replay()
    torch.cuda.synchronize()
    assert two[2].tolist() == [65, 46] and torch.equal(O, O3) and torch.equal(two[1], want[1])
    kv = rnd((1, 1, 50, d), 6)
    acc = rnd((1, 1, 50), 7).float()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        keep, lens = sdpa.evict(kv, kv.clone(), acc, i32([50]), 10)
    side.synchronize()
    assert lens.tolist() == [10] and (acc[0, 0, 10:] == 0).all()
