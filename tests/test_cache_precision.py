"""How far decodes over the bounded cache may be off, held so tightly that the loss of a few bits shows.

Values come in pairs of opposite sign whose keys are nearly the same, so an output is small beside what it is the sum of, and its own
rounding to bf16 hides nothing.  With p the weights and e the half step of what enters the sum of values (2^-12 for p s in
4-bit caches, 2^-17 for p in two bf16 parts), roundings of different keys are independent: their sum is within six times
e / sqrt(3) times the root of the sum of (p v)^2, with s c for v in 4 bits.  Scores are off by delta = (d / 16 + 8) 2^-23 |q|_2 |k|_2 |scale| (a unit per
16 products and eight more), the LSE by its keys' deltas and 2^-20 (1 + |LSE|), weights by both.

That the check is tight enough is tested on the CPU, with mistakes in the results that it is given.
"""
import math

import pytest

torch = pytest.importorskip("torch")


def inputs(bits, B, Hkv, G, n, d, seed):
    """q, keys, values, |keys| and |values| as their products add up, the part of the values whose products with p are rounded, all in
    64 bits, and the cache's arrays (on the CPU)."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, dtype=torch.float64)
    q = (0.3 * normal(B, Hkv * G, d)).to(torch.bfloat16)
    if bits == 16:
        k = normal(B, Hkv, n, d)
        k[:, :, 1::2] = k[:, :, 0:n - 1:2][:, :, :n // 2] + 0.05 * normal(B, Hkv, n // 2, d)
        v = normal(B, Hkv, n, d)
        v[:, :, 1::2] = -v[:, :, 0:n - 1:2][:, :, :n // 2]
        cache = [k.to(torch.bfloat16), v.to(torch.bfloat16)]
        k, v = (t.double() for t in cache)
        return q, k, v, k.abs(), v.abs(), v, cache
    ng, cache, out = d // 32, [], []
    ch = torch.arange(d)
    byte, shift = 2 * (ch % 32 // 4 * ng + ch // 32) + ch % 4 // 2, 4 * (ch % 2)
    for name in "kv":
        # scales of four bits, so that the minimum -7.5 s is exact and 15 - c stands for the negative
        s = 2.0 ** torch.randint(-3, 0, (B, Hkv, n, ng), generator=gen).double() * (1 + torch.randint(0, 8, (B, Hkv, n, ng), generator=gen) / 8)
        c = torch.randint(0, 16, (B, Hkv, n, d), generator=gen)
        s[:, :, 1::2] = s[:, :, 0:n - 1:2][:, :, :n // 2]
        pair = c[:, :, 0:n - 1:2][:, :, :n // 2]
        near = torch.randint(0, 40, pair.shape, generator=gen) == 0  # now and then a key's code is one off
        c[:, :, 1::2] = 15 - pair if name == "v" else (pair + near).clamp_max(15)
        codes = torch.zeros((B, Hkv, n, d // 2), dtype=torch.int64)
        codes.index_add_(-1, byte, c << shift)
        wide = s.repeat_interleave(32, -1)
        out += [wide * (c - 7.5), wide * c + 7.5 * wide, wide * c]
        cache += [codes.to(torch.uint8), torch.stack((s, -7.5 * s), -1).to(torch.bfloat16)]
    return q, out[0], out[3], out[1], out[4], out[5], cache


def softmax64(q, k, scale):
    B, Hkv, n, d = k.shape
    s = q.double().view(B, Hkv, -1, d) @ k.transpose(-1, -2) * scale
    return s, torch.softmax(s, -1), torch.logsumexp(s, -1)


def check(bits, q, k, v, k_abs, v_abs, v_part, scale, O, L, W):
    B, Hkv, n, d = k.shape
    _, p, lse = softmax64(q, k, scale)
    qq = q.double().view(B, Hkv, -1, d)
    delta = (d / 16 + 8) * 2.0 ** -23 * qq.norm(dim=-1)[..., None] * k_abs.norm(dim=-1)[:, :, None] * abs(scale)
    of_lse = (p * delta).sum(-1) + 2.0 ** -20 * (1 + lse.abs())
    rel = delta + of_lse[..., None]
    want = p @ v
    assert ((L.double().view(B, Hkv, -1) - lse).abs() <= of_lse).all(), "LSE"
    assert ((W.double() - p.sum(2)).abs() <= (rel * p).sum(2) + 2.0 ** -22 * p.sum(2)).all(), "weights"
    half = 2.0 ** -12 if bits == 4 else 2.0 ** -17
    allowed = 2.0 ** -8 * want.abs() + 6 * half / math.sqrt(3) * ((p * p) @ (v_part * v_part)).sqrt() + (p * rel) @ v_abs
    err = (O.double().view(B, Hkv, -1, d) - want).abs()
    assert (err <= allowed).all(), "outputs"


SHAPES = [(1, 1, 1, 48, 64), (2, 2, 4, 48, 128), (1, 2, 12, 97, 64), (1, 1, 16, 48, 128), (1, 2, 3, 1000, 128), (1, 1, 8, 4099, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,G,n,d", SHAPES)
@pytest.mark.parametrize("bits", [4, 16])
def test_decode(cuda_device, bits, B, Hkv, G, n, d):
    import memory_optimal_sdpa_b200 as sdpa
    q, *exact, cache = inputs(bits, B, Hkv, G, n, d, n + d)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    acc = torch.zeros((B, Hkv, n), device="cuda")
    c = [t.cuda() for t in cache]
    O, L = sdpa.decode_kv4(q.cuda(), sdpa.Kv4Cache(*c), lens, acc=acc) if bits == 4 else sdpa.decode_acc(q.cuda(), *c, lens, acc)
    check(bits, q, *exact, d ** -0.5, O.cpu(), L.cpu(), acc.cpu())


# ------------------------------------------------------------------------------------------ the check itself
def results(q, k, v, v_part, scale, of_scores=None, of_weights=None, of_products=None, drop=None):
    """O, LSE and weights with a mistake: a function of the scores, of the weights that multiply values, or a key left out of one of them."""
    B, Hkv, n, d = k.shape
    s, p, lse = softmax64(q, k, scale)
    if of_scores:
        s = of_scores(s)
        p, lse = torch.softmax(s, -1), torch.logsumexp(s, -1)
    W, used = p.sum(2), p
    if of_weights:  # on weights up to 1, as a running softmax has them
        top = p.amax(-1, keepdim=True)
        used = of_weights(p / top) * top
    if drop == "values":
        used = used.clone()
        used[..., n // 2] = 0
    if drop == "weights":
        W = W.clone()
        W[..., n // 2] = 0
    if drop == "keys":
        s = s.clone()
        s[..., n // 2] = -math.inf
        used, lse = torch.softmax(s, -1), torch.logsumexp(s, -1)
    O = used @ v_part + (p if drop is None else used) @ (v - v_part)
    return O.float().to(torch.bfloat16).view(B, -1, d), lse.float().view(B, -1), W.float()


def one_part(x):
    return x.to(torch.bfloat16).double()


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("B,Hkv,G,n,d", SHAPES)
def test_right_results_pass(bits, B, Hkv, G, n, d):
    q, *exact, _ = inputs(bits, B, Hkv, G, n, d, n + d)
    check(bits, q, *exact, d ** -0.5, *results(q, exact[0], exact[1], exact[4], d ** -0.5))
    if bits == 4:  # p s in fp16 is what is allowed
        check(bits, q, *exact, d ** -0.5, *results(q, exact[0], exact[1], exact[4], d ** -0.5, of_weights=lambda p: p.half().double()))


@pytest.mark.parametrize("mistake", [dict(of_weights=one_part), dict(of_scores=lambda s: s.half().double()), dict(of_scores=lambda s: s.to(torch.bfloat16).double()),
                                     dict(drop="values"), dict(drop="weights"), dict(drop="keys"), dict(of_scores=lambda s: s * (1 + 2.0 ** -13))])
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("B,Hkv,G,n,d", SHAPES[:5])
def test_mistakes_do_not(bits, B, Hkv, G, n, d, mistake):
    q, *exact, _ = inputs(bits, B, Hkv, G, n, d, n + d)
    with pytest.raises(AssertionError):
        check(bits, q, *exact, d ** -0.5, *results(q, exact[0], exact[1], exact[4], d ** -0.5, **mistake))
